"""The launch rules of the norm and of the router's training (csrc/plan.hpp), built for the CPU with g++."""
from __future__ import annotations

import ctypes
import functools
import os
import random
import subprocess
import tempfile

from tests.planlib import HEADER

SOURCE = """
#include "%s"
using namespace fp8q;
extern "C" void norm(int64_t rows, int64_t cols, int64_t* out) {
    const NormShape n = pick_norm(rows, cols);
    out[0] = n.waves; out[1] = n.chunks; out[2] = norm_fits(rows, cols);
}
extern "C" void back(int64_t rows, int64_t cols, int64_t* out) {
    const NormBackPlan p = pick_norm_back(rows, cols);
    out[0] = p.waves; out[1] = p.chunks; out[2] = p.rows; out[3] = p.blocks;
}
extern "C" void route(int64_t T, int64_t E, int64_t S, int64_t* out) {
    out[0] = route_lanes(E); out[1] = balance_rows(T, E); out[2] = balance_slots(T, E, S); out[3] = balance_groups(T, E, S);
}
"""


@functools.lru_cache(None)
def rules():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SOURCE % HEADER)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wno-unused-function", "-Werror", "-shared", "-fPIC", src, "-o", lib], check=True)
        return ctypes.CDLL(lib)


def ask(name, *args):
    out = (ctypes.c_int64 * 4)()
    getattr(rules(), name)(*(ctypes.c_int64(a) for a in args), out)
    return list(out)


# the kernels that the library has
SHAPES = {(1, 1), (1, 2), (1, 4), (2, 4), (4, 4), (8, 4), (16, 4), (16, 1)}


def test_registers_hold_every_row():
    rng = random.Random(1)
    for _ in range(20000):
        rows, cols = int(2 ** rng.uniform(0, 24)), int(2 ** rng.uniform(0, 17))
        waves, chunks, fits, _ = ask("norm", rows, cols)
        if cols < 8 or cols > 32768:
            assert chunks == 0
        else:
            assert (waves, chunks) in SHAPES and cols <= 512 * waves * chunks
        threads = -(-rows // (max(4, waves) // waves if chunks else 1)) * 64 * max(4, waves)
        assert bool(fits) == (threads < 1 << 32)
        waves, chunks, at_a_time, blocks = ask("back", rows, cols)
        assert blocks <= 256 and blocks <= rows and 1 <= waves * at_a_time <= 16
        assert chunks == 0 or (chunks in (1, 2) and cols <= 512 * waves * chunks)
        groups = -(-rows // at_a_time)
        assert blocks * -(-groups // blocks) < groups + blocks  # no block takes a turn more than it must
    assert ask("back", 0, 64)[3] == 0


def test_documented_rows_are_taken():
    for cols in (1, 7, 8, 512, 513, 1024, 2048, 4096, 8192, 32769, 1 << 20):
        assert ask("norm", (1 << 24) - 1, cols)[2]
    for cols in (8193, 16384, 16385, 32768):
        assert ask("norm", (1 << 22) - 1, cols)[2]


def test_chunks_of_the_balance():
    rng = random.Random(2)
    for _ in range(20000):
        T, E, S = int(2 ** rng.uniform(0, 30)), rng.randint(1, 1024), int(2 ** rng.uniform(0, 20))
        lanes, rows, slots, groups = ask("route", T, E, S)
        assert groups == 1 or (groups <= 64 and groups == -(-E // 32))  # (a wave adds them)
        assert lanes in (1, 2, 4, 8, 16, 32, 64) and 16 * lanes >= E and (lanes == 1 or 8 * lanes < E)
        chunks = -(-T // rows)
        assert chunks <= 512 and slots == chunks + S  # chunk c and sequence s share place c + s: c < chunks, s < S


def test_few_tokens_need_no_workspace():
    import fp8_quantization_grouped_amd as fq
    for E in (1, 8, 16, 17, 64, 65, 300, 1024):
        once = ask("route", 1, E, 1)[1]
        assert fq.moe_balance_workspace_size(once, E, 5) == 0
        assert fq.moe_balance_workspace_size(once + 1, E, 5) == (2 + 5) * E * 8
