"""Block-scaled FP8 and the few-token layer without a GPU: the 64-bit arithmetic that the GPU tests
compare with, and the C entry points' refusals (no call here gets past its argument checks)."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest
import torch

import oracle
import workloads
from tests import blocklib as bl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "fp8_quantization_grouped_amd", "libfp8qg.so")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


# ------------------------------------------------------------- the arithmetic compared with

def bits(x):
    return x.view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("rows", [1, 7, 64])
def test_one_block_is_the_rowwise_oracle(rows):
    """128 columns are one block: the rowwise quantizer's bytes, and one over its scale."""
    x = torch.randn(rows, 128, generator=torch.Generator().manual_seed(rows)).to(torch.bfloat16)
    x[rows // 2, 5] = 300.0
    q, d = bl.quant_rowwise(x)
    oq, os_ = oracle.quant_rowwise(bits(x), 1)
    assert np.array_equal(q.numpy(), oq)
    assert np.array_equal(d[0].float().numpy(), np.float32(1.0) / os_)


def test_blocks_are_independent_and_square_blocks_are_transposable():
    x = torch.randn(200, 300, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    q, d = bl.quant_rowwise(x)
    for b in range(3):
        qb, db = bl.quant_rowwise(x[:, 128 * b:128 * (b + 1)])
        assert torch.equal(q[:, 128 * b:128 * (b + 1)], qb) and torch.equal(d[b], db[0])
    qt, dt = bl.quant_colwise(x)
    q2, d2 = bl.quant_rowwise(x.t().contiguous())
    assert torch.equal(qt, q2) and torch.equal(dt, d2)
    q, d = bl.quant_square(x)
    q2, d2 = bl.quant_square(x.t().contiguous())
    assert torch.equal(q.t(), q2) and torch.equal(d.t(), d2)


def test_grid_is_every_code():
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    v = bl.decode(codes)
    assert torch.equal(bl.to_bytes(bl.grid(v)), codes)
    # halfway between two neighbours goes to the even code, a hair to either side to that side
    pos = v[(codes < 0x7F)]
    mid = (pos[:-1] + pos[1:]) / 2
    even = torch.where(torch.arange(len(mid)) % 2 == 0, pos[:-1], pos[1:])
    assert torch.equal(bl.grid(mid), even)
    assert torch.equal(bl.grid(mid * (1 + 1e-9)), pos[1:]) and torch.equal(bl.grid(mid * (1 - 1e-9)), pos[:-1])


# ------------------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def fn():
    if not os.path.exists(LIB):
        pytest.fail(f"{LIB} not built (run __graft_entry__.build())")
    import fp8_quantization_grouped_amd as fq
    lib = ctypes.CDLL(LIB)

    def get(name):
        f = getattr(lib, name)
        f.restype, f.argtypes = fq.SIGNATURES[name]
        return f

    return get


P = ctypes.c_void_p(4096)  # aligned, never dereferenced


def refuse(f, good, changes):
    """Each change of the good arguments gives its status; a change is {position: value, ..}."""
    for change, status in changes:
        args = list(good)
        for at, value in change.items():
            args[at] = value
        assert f(*args) == status, (change, status)


def test_quantizers_refuse(fn):
    good = [P, 4, 256, 256, P, 256, P, 4, None]
    refuse(fn("fp8_block_quant_rowwise"), good, [
        ({1: -1}, INVALID), ({2: -1}, INVALID), ({3: 255}, INVALID), ({5: 255}, INVALID), ({7: 3}, INVALID),
        ({0: None}, INVALID), ({4: None}, INVALID), ({6: None}, INVALID), ({1: 0}, OK), ({2: 0}, OK)])
    good = [P, 4, 256, 256, P, 256, P, 4, P, 4, P, 256, None]
    refuse(fn("fp8_block_quant_dual"), good, [
        ({1: -1}, INVALID), ({3: 255}, INVALID), ({5: 255}, INVALID), ({7: 3}, INVALID), ({9: 3}, INVALID), ({11: 255}, INVALID),
        ({0: None}, INVALID), ({4: None}, INVALID), ({6: None}, INVALID), ({8: None}, INVALID), ({10: None}, INVALID), ({1: 0}, OK), ({2: 0}, OK)])
    good = [P, 2, 64, 256, 256, P, 256, P, 128, P, None]
    refuse(fn("fp8_block_quant_weights"), good, [
        ({1: -1}, INVALID), ({2: -1}, INVALID), ({4: 255}, INVALID), ({6: 255}, INVALID), ({8: 127}, INVALID),
        ({0: None}, INVALID), ({9: None}, INVALID), ({5: None, 7: None}, INVALID), ({1: 65536, 8: 1 << 40}, UNSUPPORTED), ({1: 0}, OK), ({2: 0}, OK)])


def test_product_refuses(fn):
    f = fn("fp8_block_grouped_gemm")
    M, N, K, G = 32, 64, 256, 2
    #       0  1  2  3  4  5  6  7      8  9  10 11 12 13 14 15 16 17 18 19 20 21   22
    good = [0, P, K, P, M, P, K, N * K, P, 2, 1, 2, P, G, M, N, K, P, N, 0, P, 256, None]
    refuse(f, good, [
        ({0: 2}, INVALID), ({13: 0}, INVALID), ({12: None}, INVALID), ({14: -1}, INVALID), ({15: -1}, INVALID), ({16: -1}, INVALID),
        ({2: K - 16}, INVALID), ({6: K - 16}, INVALID), ({4: M - 1}, INVALID), ({18: N - 1}, INVALID), ({19: 2}, INVALID),
        ({7: -16}, INVALID), ({9: -1}, INVALID), ({10: -1}, INVALID), ({11: -1}, INVALID),
        ({1: None}, INVALID), ({3: None}, INVALID), ({5: None}, INVALID), ({8: None}, INVALID), ({17: None}, INVALID),
        ({21: 255}, WORKSPACE), ({20: ctypes.c_void_p(4098)}, INVALID), ({17: ctypes.c_void_p(4097)}, INVALID),
        ({3: ctypes.c_void_p(4098)}, INVALID), ({1: ctypes.c_void_p(4104)}, UNSUPPORTED), ({5: ctypes.c_void_p(4104)}, UNSUPPORTED),
        ({16: 248}, UNSUPPORTED), ({2: K + 8}, UNSUPPORTED), ({6: K + 8}, UNSUPPORTED), ({7: N * K + 8}, UNSUPPORTED),
        ({13: 2049}, UNSUPPORTED), ({14: 1 << 31, 4: 1 << 31}, UNSUPPORTED), ({2: 1 << 24}, UNSUPPORTED), ({18: 1 << 24}, UNSUPPORTED),
        ({9: 1 << 30}, UNSUPPORTED), ({13: 2048, 14: 1 << 30, 4: 1 << 30}, UNSUPPORTED), ({14: 0}, OK), ({15: 0}, OK)])
    #       wgrad: a [K][M], b [N][M]
    good = [1, P, M, P, K, P, M, 0, P, 1, N, 0, P, G, M, N, K, P, N, 0, P, 256, None]
    refuse(f, good, [
        ({7: 16}, INVALID), ({11: 1}, INVALID), ({9: 2}, INVALID), ({10: N - 1}, INVALID), ({4: K - 1}, INVALID),
        ({2: M - 1}, INVALID), ({2: M + 8}, UNSUPPORTED), ({6: M + 8}, UNSUPPORTED), ({16: 0}, OK), ({15: 0}, OK)])


def test_route_refuses(fn):
    f, ws = fn("moe_route"), fn("moe_route_workspace_size")
    T, H, E = 4, 4096, 64
    assert ws(T, H, E) >= T * E * 4 and ws(0, H, E) == 256
    #       0  1  2  3  4  5  6  7     8  9  10 11   12 13 14 15         16
    good = [P, T, H, H, P, E, H, None, 0, 8, 1, 1.0, P, P, P, ws(T, H, E), None]
    refuse(f, good, [
        ({1: -1}, INVALID), ({2: 0}, INVALID), ({5: 0}, INVALID), ({3: H - 8}, INVALID), ({6: H - 8}, INVALID), ({8: 2}, INVALID),
        ({9: 0}, INVALID), ({9: E + 1}, INVALID), ({0: None}, INVALID), ({4: None}, INVALID), ({12: None}, INVALID), ({13: None}, INVALID),
        ({9: 33}, UNSUPPORTED), ({5: 1025}, UNSUPPORTED), ({2: H - 4}, UNSUPPORTED), ({3: H + 4}, UNSUPPORTED), ({6: H + 4}, UNSUPPORTED),
        ({0: ctypes.c_void_p(4104)}, UNSUPPORTED), ({4: ctypes.c_void_p(4104)}, UNSUPPORTED), ({1: 1 << 21}, UNSUPPORTED),
        ({14: None}, WORKSPACE), ({15: ws(T, H, E) - 1}, WORKSPACE), ({14: ctypes.c_void_p(4098)}, INVALID), ({1: 0}, OK)])


def test_layer_refuses(fn):
    f, ws = fn("fp8_moe_few_tokens"), fn("fp8_moe_few_tokens_workspace_size")
    T, H, I, E, k = 4, 256, 128, 8, 2
    size = ws(T, H, I, k)
    assert size >= T * k * (H + I) * 4 and ws(0, H, I, k) == 256
    #       0  1  2  3  4  5  6  7  8  9          10 11 12 13 14 15 16     17 18 19 20 21 22 23 24 25 26    27
    good = [P, T, H, H, P, P, k, P, H, 2 * I * H, P, 2, 1, 4, P, I, H * I, P, 1, 1, 2, E, I, P, H, P, size, None]
    refuse(f, good, [
        ({1: -1}, INVALID), ({2: 0}, INVALID), ({22: 0}, INVALID), ({21: 0}, INVALID), ({6: 0}, INVALID), ({3: H - 8}, INVALID),
        ({8: H - 16}, INVALID), ({15: I - 16}, INVALID), ({24: H - 1}, INVALID), ({9: -16}, INVALID), ({16: -16}, INVALID),
        ({11: -1}, INVALID), ({20: -1}, INVALID), ({0: None}, INVALID), ({4: None}, INVALID), ({5: None}, INVALID), ({7: None}, INVALID),
        ({10: None}, INVALID), ({14: None}, INVALID), ({17: None}, INVALID), ({23: None}, INVALID),
        ({1: 129}, UNSUPPORTED), ({21: 1025}, UNSUPPORTED), ({6: 33}, UNSUPPORTED), ({2: H - 8}, UNSUPPORTED), ({22: I - 8, 15: I}, UNSUPPORTED),
        ({3: H + 4}, UNSUPPORTED), ({8: H + 8}, UNSUPPORTED), ({15: I + 8}, UNSUPPORTED), ({9: 2 * I * H + 8}, UNSUPPORTED),
        ({0: ctypes.c_void_p(4104)}, UNSUPPORTED), ({7: ctypes.c_void_p(4104)}, UNSUPPORTED), ({14: ctypes.c_void_p(4104)}, UNSUPPORTED),
        ({8: 1 << 26}, UNSUPPORTED), ({3: 1 << 28}, UNSUPPORTED), ({25: None}, WORKSPACE), ({26: size - 1}, WORKSPACE), ({25: ctypes.c_void_p(4104)}, INVALID), ({1: 0}, OK)])


def test_binding_refuses_host_tensors():
    import fp8_quantization_grouped_amd as fq
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q, d = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(2, 4)
    for bad in (lambda: fq.fp8_block_quant_rowwise(x), lambda: fq.fp8_block_quant_dual(x), lambda: fq.fp8_block_quant_weights(x, 2),
                lambda: fq.fp8_block_grouped_gemm(0, q, d, q[None], d), lambda: fq.moe_route(x, x, 2),
                lambda: fq.fp8_moe_few_tokens(x, d.int(), d, q[None], d, q[None], d)):
        with pytest.raises(ValueError):
            bad()


def test_small_router_takes_no_workspace(fn):
    f, ws = fn("moe_route"), fn("moe_route_workspace_size")
    assert ws(4, 256, 4) == 0 and ws(4, 2048, 64) > 0
    #       0  1  2    3    4  5  6    7     8  9  10 11   12 13 14    15 16
    refuse(f, [P, 4, 2048, 2048, P, 64, 2048, None, 0, 2, 1, 1.0, P, P, None, 0, None], [({1: 0}, OK), ({}, WORKSPACE)])
