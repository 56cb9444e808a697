"""The launch rules of the block-scaled kernels (csrc/plan.hpp), built for the CPU with g++."""
from __future__ import annotations

import ctypes
import functools
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "fp8_quantization_grouped_amd", "csrc", "plan.hpp")
TILES = ["64x64", "128x64", "128x128", "256x256"]

SOURCE = """
#include "%s"
extern "C" int tile(int fwd, int64_t M, int64_t N, int64_t K, int64_t G, int64_t cus) {
    return fp8q::pick_block_tile(fwd != 0, M, N, K, G, cus);
}
extern "C" void stream(int down, int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int64_t cus, int* out) {
    const fp8q::StreamPlan p = fp8q::pick_stream(down != 0, T, k, E, H, I, cus);
    out[0] = p.mt; out[1] = p.pass; out[2] = p.parts;
}
"""


@functools.lru_cache(None)
def rules():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SOURCE % HEADER)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wno-unused-function", "-Werror", "-shared", "-fPIC", src, "-o", lib], check=True)
        L = ctypes.CDLL(lib)
    i64, i = ctypes.c_int64, ctypes.c_int
    L.tile.argtypes = [i, i64, i64, i64, i64, i64]
    L.stream.argtypes = [i, i64, i64, i64, i64, i64, i64, ctypes.POINTER(i)]
    return L


def tile(fwd, M, N, K, G, cus=256):
    """Output tile of the product's launch."""
    return TILES[rules().tile(int(fwd), M, N, K, G, cus)]


def stream(down, T, top_k, E, H, I, cus=256):
    """(token tiles of 16 in a pass, tokens of a pass, parts of the contraction) of one of the layer's products."""
    out = (ctypes.c_int * 3)()
    rules().stream(int(down), T, top_k, E, H, I, cus, out)
    return tuple(out)
