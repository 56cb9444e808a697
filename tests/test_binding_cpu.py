"""What the binding of the block-scaled operators hands to the C entry points, without a GPU: host
tensors that say they are on one, and a library that records its calls instead of making them."""
from __future__ import annotations

import pytest
import torch

import fp8_quantization_grouped_amd as fq


class OnGpu(torch.Tensor):
    """A host tensor that passes the binding's device checks."""
    is_cuda = property(lambda self: True)


def gpu(t):
    return t.as_subclass(OnGpu)


def zeros(*shape, dtype=torch.float32):
    return gpu(torch.zeros(*shape, dtype=dtype))


class Recorder:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_size") or name.endswith("status_string"):
            return getattr(self.real, name)
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def calls(monkeypatch):
    r = Recorder(fq.lib())
    monkeypatch.setattr(fq, "_lib", r)
    monkeypatch.setattr(fq, "_device_now", lambda: None)
    monkeypatch.setattr(fq, "_raw_stream", lambda index: 0)
    return r.calls


BF16, U8, F32 = torch.bfloat16, torch.uint8, torch.float32


# --------------------------------------- rows that overlap: the C checks have to see their stride

def overlapping(rows, cols, dtype=F32, stride=0):
    """[rows, cols] of one row's storage (stride 0), or of rows that begin stride apart."""
    return gpu(torch.zeros(cols + stride * (rows - 1), dtype=dtype).as_strided((rows, cols), (stride, 1)))


@pytest.mark.parametrize("stride", [0, 3])
def test_overlapping_factors_of_a_product_reach_its_checks(calls, stride):
    M, N, K, G = 64, 32, 512, 2
    off = zeros(G, dtype=torch.int32)
    fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, zeros(M, K, dtype=U8), overlapping(4, M, stride=stride),
                              zeros(G, N, K, dtype=U8), zeros(G, 1, 4), off)
    assert calls[-1][1][4] == stride < M  # ld_sa: refused
    fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, zeros(K, 512, dtype=U8), zeros(4, K), zeros(N, 512, dtype=U8),
                              overlapping(4, N, stride=stride), off)
    assert calls[-1][1][10] == stride < N  # sb_k: refused
    fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, zeros(K, 512, dtype=U8), overlapping(4, K, stride=stride),
                              zeros(N, 512, dtype=U8), zeros(4, N), off)
    assert calls[-1][1][4] == stride < K


@pytest.mark.parametrize("stride", [0, 3])
def test_overlapping_outputs_of_the_quantizers_reach_their_checks(calls, stride):
    x = zeros(300, 256, dtype=BF16)
    for kw, at in (({"s_rows": overlapping(2, 300, stride=stride)}, 7), ({"q_t": overlapping(256, 300, U8, stride)}, 9),
                   ({"s_cols": overlapping(3, 256, stride=stride)}, 11), ({"q": overlapping(300, 256, U8, stride)}, 5)):
        fq.fp8_block_quant_dual(x, **kw)
        assert calls[-1][1][at] == stride, kw.keys()
    fq.fp8_block_quant_weights(x, 3, q_t=overlapping(256, 300, U8, stride))
    assert calls[-1][1][8] == stride


@pytest.mark.parametrize("stride", [0, 1])
def test_overlapping_gradients_of_one_row_each_reach_the_checks(calls, stride):
    """[groups, 1, N] with the groups on top of each other."""
    G, N = 3, 32
    c = gpu(torch.zeros(64, dtype=BF16).as_strided((G, 1, N), (stride, stride, 1)))
    fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, zeros(1, 128, dtype=U8), zeros(1, 1), zeros(N, 128, dtype=U8), zeros(1, N),
                              zeros(G, dtype=torch.int32), c=c)
    assert calls[-1][1][18] == stride < N  # ldc


def test_ordinary_strides_are_handed_on(calls):
    M, N, K, G = 64, 32, 512, 2
    off = zeros(G, dtype=torch.int32)
    wide = zeros(4, M + 6)[:, :M]
    c = zeros(M, N + 5, dtype=BF16)[:, :N]
    fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, zeros(M, K, dtype=U8), wide, zeros(G, N, K, dtype=U8), zeros(G, 1, 4), off, c=c)
    assert calls[-1][1][4] == M + 6 and calls[-1][1][18] == N + 5
    c = zeros(G, K, N + 5, dtype=F32)[:, :, :N]
    fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, zeros(K, 512, dtype=U8), zeros(4, K), zeros(N, 512, dtype=U8),
                              zeros(4, N + 3)[:, :N], off, c=c)
    assert calls[-1][1][10] == N + 3 and calls[-1][1][18] == N + 5
    one = gpu(torch.zeros(N, dtype=F32).as_strided((1, N), (1, 1)))  # one row: its stride says nothing
    fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, zeros(K, 128, dtype=U8), zeros(1, K), zeros(N, 128, dtype=U8), one, off)
    assert calls[-1][1][10] >= N
    fq.fp8_block_quant_dual(zeros(0, 256, dtype=BF16))
    fq.fp8_block_quant_dual(zeros(5, 0, dtype=BF16))
    args = calls[-1][1]
    assert args[7] >= 5 and args[9] >= 5 and args[11] >= 0


# ------------------------------------------------------------------------ workspaces of the caller

def moe_args(T=4, H=256, I=128, E=3, k=2):
    return (zeros(T, H, dtype=BF16), zeros(T, k, dtype=torch.int32), zeros(T, k), zeros(E, 2 * I, H, dtype=U8),
            zeros(E, 2 * I // 128, 2), zeros(E, H, I, dtype=U8), zeros(E, 2, 1))


def with_workspace(kind, ws):
    if kind == "product":
        return fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, zeros(4, 256, dtype=U8), zeros(2, 4), zeros(1, 8, 256, dtype=U8),
                                         zeros(1, 1, 2), workspace=ws)
    if kind == "route":
        return fq.moe_route(zeros(4, 4096, dtype=BF16), zeros(64, 4096, dtype=BF16), 2, workspace=ws)
    return fq.fp8_moe_few_tokens(*moe_args(), workspace=ws)


@pytest.mark.parametrize("kind", ["product", "route", "layer"])
def test_workspaces_are_checked(calls, kind):
    n = 1 << 16
    for bad in (torch.zeros(n, dtype=U8),                       # host memory
                zeros(1, dtype=U8).expand(n),                   # one byte that says it is many
                zeros(2 * n, dtype=U8)[::2],
                gpu(torch.zeros(n, dtype=U8, device="meta"))):  # another device
        with pytest.raises(ValueError, match="workspace"):
            with_workspace(kind, bad)
    assert calls == []
    with_workspace(kind, zeros(n, dtype=U8))
    with_workspace(kind, zeros(n // 4))  # any type
    with_workspace(kind, zeros(8, n // 8, dtype=U8))
    assert len(calls) == 3 and all(n in args for _, args in calls)


# -------------------------------------------------- one row: whatever its stride, it is no limit

def one_row(cols, stride, dtype):
    return gpu(torch.zeros(cols, dtype=dtype).as_strided((1, cols), (stride, 1)))


@pytest.mark.parametrize("stride", [1, 256, 257, 4097, 1 << 25, 1 << 34, 1 << 58])
def test_one_row_of_any_stride(calls, stride):
    """A token cut out of a longer buffer ([:1], or [:, -1] of a batch of one)."""
    H, I, E, k = 256, 128, 3, 2
    x = one_row(H, stride, BF16)
    fq.moe_route(x, zeros(E, H, dtype=BF16), k)
    assert calls[-1][1][3] == H
    _, ids, weights, *w = moe_args(1, H, I, E, k)
    fq.fp8_moe_few_tokens(x, ids, weights, *w, y=one_row(H, stride, BF16))
    assert calls[-1][1][3] == H and calls[-1][1][24] == H
    fq.fp8_block_quant_rowwise(x)
    assert calls[-1][1][3] == H
    a, b = one_row(H, stride, U8), gpu(torch.zeros(H, dtype=U8).as_strided((1, 1, H), (stride, stride, 1)))
    fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, a, zeros(2, 1), b, zeros(1, 1, 2), c=one_row(1, stride, F32))
    args = calls[-1][1]
    assert args[2] == H and args[6] == H and args[7] == 0 and args[18] in (1, 16)
    fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, a, zeros(2, 1), a, zeros(2, 1))
    assert calls[-1][1][2] == H and calls[-1][1][6] == H


def test_one_padded_row_keeps_its_padding(calls):
    """A row of 1333 bytes whose storage goes on to 1344: the product takes it, as it takes many."""
    a = gpu(torch.zeros(1, 1344, dtype=U8))[:, :1333]
    fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, a, zeros(11, 1), a, zeros(11, 1))
    assert calls[-1][1][2] == 1344 and calls[-1][1][6] == 1344
    bare = zeros(1, 1333, dtype=U8)
    fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, bare, zeros(11, 1), a, zeros(11, 1))
    assert calls[-1][1][2] == 1333  # refused: nothing says that there are 1344 bytes


def test_a_contraction_of_length_zero_is_taken(calls):
    """The strides of tensors without elements are 1, which is no multiple of 16."""
    fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, zeros(8, 0, dtype=U8), zeros(0, 8), zeros(2, 5, 0, dtype=U8), zeros(2, 1, 0),
                              zeros(2, dtype=torch.int32))
    args = calls[-1][1]
    assert args[2] % 16 == 0 and args[6] % 16 == 0 and args[7] % 16 == 0 and args[14:17] == (8, 5, 0)


# ------------------------------------------------------------------------------- no lost gradients

def test_operands_that_require_a_gradient_are_refused(calls):
    """moe_route and the layer have no backward: a result cut from autograd is not given out silently."""
    def operands(which):
        x, ids, weights, *w = moe_args()
        t = {"x": x, "router": zeros(3, 256, dtype=BF16), "bias": zeros(3), "weights": weights}
        t[which].requires_grad_()
        return t, ids, w

    for which in ("x", "router", "bias"):
        t, _, _ = operands(which)
        route = lambda: fq.moe_route(t["x"], t["router"], 2, bias=t["bias"])
        with pytest.raises(ValueError, match="gradient"):
            route()
        with torch.no_grad():
            route()
    for which in ("x", "weights"):
        t, ids, w = operands(which)
        layer = lambda: fq.fp8_moe_few_tokens(t["x"], ids, t["weights"], *w)
        with pytest.raises(ValueError, match="gradient"):
            layer()
        with torch.inference_mode():
            layer()
    assert len(calls) == 5
