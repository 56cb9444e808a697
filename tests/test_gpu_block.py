"""Block-scaled FP8 quantizers and grouped products (blocks of 128) against 64-bit arithmetic."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import blocklib as bl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_quantization_grouped_amd as m
    m.lib()
    return m


def values(seed, rows, cols, scale=1.0, ld=None):
    """bf16 normals with outliers, a zero block and a zero row, as a strided view if ld is given."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * scale
    x = torch.where(torch.rand(rows, cols, generator=g) < 0.01, x * 50, x)
    x[: min(rows, 130), 128:256] = 0
    x[rows // 2] = 0
    x = x.to(torch.bfloat16)
    if ld is None:
        return x.to(DEV)
    full = torch.full((rows, ld), float("nan"), dtype=torch.bfloat16)
    full[:, :cols] = x
    return full.to(DEV)[:, :cols]


def same(got, want):
    assert got.shape == want.shape
    got = got.cpu()
    bad = torch.nonzero(got != want)
    assert len(bad) == 0, (len(bad), [(tuple(map(int, i)), got[tuple(i)].item(), want[tuple(i)].item()) for i in bad[:4]])


def same_f32(got, want64):
    same(got.contiguous().view(torch.int32), want64.float().contiguous().view(torch.int32))


SHAPES = [(1, 128), (1, 8), (3, 1), (7, 13), (128, 128), (129, 136), (255, 384), (257, 1000), (300, 129), (513, 264), (64, 2064)]


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rowwise(fq, rows, cols):
    x = values(rows * 7 + cols, rows, cols)
    q, d = fq.fp8_block_quant_rowwise(x)
    wq, wd = bl.quant_rowwise(x)
    same_f32(d, wd)
    same(q, wq)


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dual(fq, rows, cols):
    x = values(rows * 5 + cols, rows, cols)
    (q, d), (q_t, d_t) = fq.fp8_block_quant_dual(x)
    wq, wd = bl.quant_rowwise(x)
    same_f32(d, wd)
    same(q, wq)
    wq, wd = bl.quant_colwise(x)
    same_f32(d_t, wd)
    same(q_t, wq)
    (none, none2), (q_t2, d_t2) = fq.fp8_block_quant_dual(x, transposed_only=True)
    assert none is None and none2 is None
    assert torch.equal(q_t2, q_t) and torch.equal(d_t2, d_t)


@pytest.mark.parametrize("experts,rows,cols", [(1, 128, 128), (3, 200, 264), (2, 129, 130), (5, 8, 16), (4, 512, 256), (2, 24, 300), (1, 1, 1)])
def test_weights(fq, experts, rows, cols):
    w = values(experts + rows + cols, experts * rows, cols, 0.02)
    q, q_t, d = fq.fp8_block_quant_weights(w, experts)
    for e in range(experts):
        at = slice(e * rows, (e + 1) * rows)
        wq, wd = bl.quant_square(w[at])
        same_f32(d[e], wd)
        same(q[at], wq)
        same(q_t[:, at], wq.t())


def test_padded_rows_and_odd_strides(fq):
    """Row strides that rule the wide accesses out, outputs inside larger buffers, NaN around x."""
    for ld, cols, ld_q, ld_t in ((301, 300, 303, 99), (304, 296, 312, 104), (320, 300, 304, 112)):
        x = values(ld, 97, cols, ld=ld)
        q_all = torch.full((97, ld_q), 7, dtype=torch.uint8, device=DEV)
        t_all = torch.full((cols, ld_t), 7, dtype=torch.uint8, device=DEV)
        (q, d), (q_t, d_t) = fq.fp8_block_quant_dual(x, q=q_all[:, :cols], q_t=t_all[:, :97])
        wq, wd = bl.quant_rowwise(x)
        same(q, wq)
        same_f32(d, wd)
        wq, wd = bl.quant_colwise(x)
        same(q_t, wq)
        same_f32(d_t, wd)
        assert bool((q_all[:, cols:] == 7).all()) and bool((t_all[:, 97:] == 7).all())


def test_every_bf16_value_under_several_maxima(fq):
    """Every finite bf16 value not above a block's maximum, so that each border of the grid and the
    rounding of the product are met."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16)
    for top in (1.0, 3.0, 0.7, 1e-3, 200.0, 1.5e30, 2.0 ** -40):
        v = bits[torch.isfinite(bits.float()) & (bits.float().abs() <= torch.tensor(top).to(torch.bfloat16).float())]
        n = -(-len(v) // 127)
        x = torch.zeros(n, 128, dtype=torch.bfloat16)
        x[:, :127] = torch.nn.functional.pad(v.float(), (0, n * 127 - len(v))).to(torch.bfloat16).view(n, 127)
        x[:, 127] = top
        x = x.to(DEV)
        q, d = fq.fp8_block_quant_rowwise(x)
        wq, wd = bl.quant_rowwise(x)
        same_f32(d, wd)
        same(q, wq)


# -------------------------------------------------------------------------------- the products

def group_ends(kind, M, G, seed=0):
    r = np.random.default_rng(seed)
    if kind == "even":
        return [(g + 1) * M // G for g in range(G)]
    if kind == "empties":
        cuts = sorted(r.integers(0, M + 1, max(0, G // 2)).tolist())
        cuts = (cuts + cuts)[: G - 1]
        return sorted(cuts) + [0] * 0 + [M] * (G - len(cuts))
    return sorted(r.integers(0, M + 1, G - 1).tolist()) + [M]


def close(got, exact, mags, dtype):
    assert got.dtype == dtype and got.shape == exact.shape
    off = (got.cpu().double() - exact).abs()
    assert bool(torch.isfinite(off).all())
    over = off - bl.product_bound(exact, mags, dtype)
    # the bound is a worst case of cut-off products; the whole is held to a tenth of it
    assert float(over.max()) <= 0 if over.numel() else True
    if exact.numel() and float(exact.norm()) > 0:
        assert float(off.norm() / exact.norm()) <= torch.finfo(dtype).eps / 2 + 2.0 ** -11


FWD = [  # M, N, K, groups, ends
    (1, 16, 16, 1, "even"), (1, 128, 128, 1, "even"), (5, 1, 144, 2, "cuts"), (300, 257, 272, 3, "cuts"),
    (1000, 513, 1040, 7, "cuts"), (512, 256, 256, 4, "empties"), (777, 384, 2064, 9, "empties"), (2, 130, 4096, 5, "cuts"),
    (260, 1408, 512, 64, "cuts"), (2100, 136, 128, 1, "even")]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,G,kind", FWD)
def test_forward(fq, M, N, K, G, kind, out):
    ends = group_ends(kind, M, G, M + N)
    x = values(M + K, M, K)
    w = values(N + K, G * N, K, 0.05)
    q, d = fq.fp8_block_quant_rowwise(x)
    wq, _, wd = fq.fp8_block_quant_weights(w, G)
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    y = fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q, d, wq.unflatten(0, (G, N)), wd, off, out_dtype=out, workspace=ws)
    assert fq.gemm_offsets_status(ws) == (0, -1)
    a = bl.real_rows(q, d)
    lo = 0
    for g, hi in enumerate(ends):
        b = bl.real_square(wq[g * N:(g + 1) * N], wd[g])
        close(y[lo:hi], *bl.product(a[lo:hi], b), out)
        lo = hi


@pytest.mark.parametrize("M,N,K,G,kind", [(1, 16, 16, 1, "even"), (300, 272, 257, 3, "cuts"), (777, 2064, 384, 9, "empties")])
def test_data_gradient(fq, M, N, K, G, kind):
    """dX = dY W on the transposed bytes with the factors' transpose."""
    ends = group_ends(kind, M, G, M + N)
    dy = values(M, M, N, 1e-3)
    w = values(N + K, G * N, K, 0.05)
    q, d = fq.fp8_block_quant_rowwise(dy)
    wq, wt, wd = fq.fp8_block_quant_weights(w, G)
    wt = torch.nn.functional.pad(wt, (0, -wt.shape[1] % 16))[:, :G * N] if wt.stride(0) % 16 else wt
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    b = wt.unflatten(1, (G, N)).transpose(0, 1)
    dx = fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q, d, b, wd.transpose(1, 2), off)
    a = bl.real_rows(q, d)
    lo = 0
    for g, hi in enumerate(ends):
        close(dx[lo:hi], *bl.product(a[lo:hi], bl.real_square(wq[g * N:(g + 1) * N], wd[g]).t()), torch.bfloat16)
        lo = hi


WG = [(1, 16, 16, 1, "even"), (128, 128, 128, 1, "even"), (129, 17, 33, 2, "cuts"), (300, 257, 272, 3, "cuts"),
      (1000, 130, 300, 7, "cuts"), (777, 264, 384, 9, "empties"), (2050, 256, 512, 40, "cuts"), (3, 64, 64, 5, "cuts")]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,G,kind", WG)
def test_weight_gradient(fq, M, N, K, G, kind, out):
    ends = group_ends(kind, M, G, M + N)
    x, dy = values(M, M, K), values(M + 1, M, N, 1e-3)
    _, (xt, xd) = fq.fp8_block_quant_dual(x, transposed_only=True)
    _, (dt, dd) = fq.fp8_block_quant_dual(dy, transposed_only=True)
    for t in (xt, dt):  # the padding of the token dimension may hold any code
        torch.as_strided(t, (t.shape[0], t.stride(0)), (t.stride(0), 1))[:, M:] = 0x7F
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    dw = fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, xt, xd, dt, dd, off, out_dtype=out, workspace=ws)
    assert fq.gemm_offsets_status(ws) == (0, -1)
    a, b = bl.real_rows(xt, xd), bl.real_rows(dt, dd)
    lo = 0
    for g, hi in enumerate(ends):
        close(dw[g], *bl.product(a[:, lo:hi], b[:, lo:hi]), out)
        if hi == lo:
            assert not bool(dw[g].any())
        lo = hi


def test_gradients_are_the_products_differences(fq):
    """The two gradients against central differences of sum(Y * dY) in the dequantized operands: the
    forward is bilinear, so a difference over a step is exact up to the products' own bound."""
    M, N, K, G = 70, 48, 160, 3
    ends = [20, 20, 70]
    x, w, dy = values(1, M, K), values(2, G * N, K, 0.05), values(3, M, N)
    wq, wt, wd = fq.fp8_block_quant_weights(w, G)
    _, (xt, xd) = fq.fp8_block_quant_dual(x)
    (dq, dd), (dt, ddt) = fq.fp8_block_quant_dual(dy)
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    f32 = torch.float32
    dx = fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, dq, dd, wt.unflatten(1, (G, N)).transpose(0, 1), wd.transpose(1, 2), off, out_dtype=f32)
    dw = fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, dt, ddt, xt, xd, off, out_dtype=f32)
    X, DYr, DYc = bl.real_rows(xt, xd).t(), bl.real_rows(dq, dd), bl.real_rows(dt, ddt).t()
    W = torch.stack([bl.real_square(wq[g * N:(g + 1) * N], wd[g]) for g in range(G)])
    of = torch.tensor([next(g for g, e in enumerate(ends) if m < e) for m in range(M)])

    def loss(X, W, DY):
        return float(((X[:, None, :] * W[of]).sum(2) * DY).sum())

    for m, k in ((0, 0), (19, 159), (20, 3), (69, 128)):
        h = torch.zeros_like(X)
        h[m, k] = 0.5
        diff = loss(X + h, W, DYr) - loss(X - h, W, DYr)
        mags = float((DYr[m].abs() * W[of[m]][:, k].abs()).sum())
        assert abs(float(dx[m, k]) - diff) <= 2.0 ** -9 * mags + 1e-9
    for g, n, k in ((0, 0, 0), (2, 47, 159), (2, 5, 127), (1, 1, 1)):
        h = torch.zeros_like(W)
        h[g, n, k] = 0.5
        diff = loss(X, W + h, DYc) - loss(X, W - h, DYc)
        mags = float((DYc[of == g][:, n].abs() * X[of == g][:, k].abs()).sum())
        assert abs(float(dw[g, n, k]) - diff) <= 2.0 ** -9 * mags + 1e-9


def test_one_group_without_offsets_and_float8_views(fq):
    x, w = values(1, 100, 256), values(2, 200, 256, 0.05)
    q, d = fq.fp8_block_quant_rowwise(x)
    wq, _, wd = fq.fp8_block_quant_weights(w, 1)
    off = torch.tensor([100], dtype=torch.int32, device=DEV)
    y = fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q, d, wq[None], wd, off)
    f8 = torch.float8_e4m3fn
    assert torch.equal(y, fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q.view(f8), d, wq[None].view(f8), wd))


def test_output_view_and_bad_offsets_stay_inside(fq):
    """A strided output keeps its surroundings; bad offsets are reported and write inside c only."""
    M, N, K, G = 130, 100, 256, 2
    x, w = values(1, M, K), values(2, G * N, K, 0.05)
    q, d = fq.fp8_block_quant_rowwise(x)
    wq, _, wd = fq.fp8_block_quant_weights(w, G)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    for offs, status in (([70, 130], (0, -1)), ([140, 130], (1, 0)), ([70, 60], (1, 1)), ([-5, 130], (1, 0))):
        full = torch.full((M + 2, N + 5), 3.0, dtype=torch.bfloat16, device=DEV)
        off = torch.tensor(offs, dtype=torch.int32, device=DEV)
        fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q, d, wq.unflatten(0, (G, N)), wd, off, c=full[1:M + 1, :N], workspace=ws)
        assert fq.gemm_offsets_status(ws) == status
        assert bool((full[0] == 3).all()) and bool((full[M + 1] == 3).all()) and bool((full[:, N:] == 3).all())


def test_refusals(fq):
    x, w = values(1, 32, 256), values(2, 64, 256, 0.05)
    q, d = fq.fp8_block_quant_rowwise(x)
    wq, _, wd = fq.fp8_block_quant_weights(w, 2)
    b = wq.unflatten(0, (2, 32))
    off = torch.tensor([10, 32], dtype=torch.int32, device=DEV)
    run = fq.fp8_block_grouped_gemm
    F = fq.GEMM_FWD_MGROUPED
    for bad in (lambda: fq.fp8_block_quant_rowwise(x.float()), lambda: fq.fp8_block_quant_rowwise(x.t()),
                lambda: fq.fp8_block_quant_rowwise(x.cpu()), lambda: fq.fp8_block_quant_rowwise(x, scales=d[:1]),
                lambda: fq.fp8_block_quant_weights(w, 3), lambda: run(7, q, d, b, wd, off), lambda: run(F, q, d[:1], b, wd, off),
                lambda: run(F, q, d, b, wd[:1], off), lambda: run(F, q, d, b, wd.double(), off), lambda: run(F, q, d, b, wd, off.long()),
                lambda: run(F, q, d, b, wd, off[:1]), lambda: run(F, q, d, b[:, :, :128], wd, off), lambda: run(F, q, d, b, wd, off, out_dtype=torch.float16),
                lambda: run(F, q, d, b, wd, off, c=torch.empty(32, 31, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises((ValueError, KeyError)):
            bad()
    with pytest.raises(RuntimeError, match="workspace"):
        run(F, q, d, b, wd, off, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(RuntimeError, match="unsupported"):
        run(F, q[:, :200], d, b[:, :, :200], wd, off)


def test_empty_sizes(fq):
    for rows, cols in ((0, 256), (5, 0)):
        x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
        q, d = fq.fp8_block_quant_rowwise(x)
        assert q.shape == (rows, cols) and d.shape == (-(-cols // 128), rows)
        fq.fp8_block_quant_dual(x)
    w = values(2, 64, 256, 0.05)
    wq, _, wd = fq.fp8_block_quant_weights(w, 2)
    q, d = fq.fp8_block_quant_rowwise(torch.empty(0, 256, dtype=torch.bfloat16, device=DEV))
    off = torch.zeros(2, dtype=torch.int32, device=DEV)
    y = fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q, d, wq.unflatten(0, (2, 32)), wd, off)
    assert y.shape == (0, 32)
    # no tokens: the weight gradient is all zeros
    e = torch.empty(48, 0, dtype=torch.uint8, device=DEV)
    s = torch.empty(0, 48, dtype=torch.float32, device=DEV)
    dw = fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, e, s, e, s, off)
    assert dw.shape == (2, 48, 48) and not bool(dw.any())


def test_other_stream_and_graph(fq):
    """On a stream of the caller's, and captured into a graph that is replayed with eager work between."""
    M, N, K, G = 200, 256, 512, 3
    w = values(2, G * N, K, 0.05)
    wq, _, wd = fq.fp8_block_quant_weights(w, G)
    b = wq.unflatten(0, (G, N))
    off = torch.tensor([50, 50, 200], dtype=torch.int32, device=DEV)
    xs = [values(s, M, K) for s in range(4)]

    def step(x):
        q, d = fq.fp8_block_quant_rowwise(x)
        return fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q, d, b, wd, off)

    want = [step(x) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(xs[1])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[1])
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step(x)
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        assert torch.equal(step(xs[(i + 1) % 4]), want[(i + 1) % 4])


def test_sizes_past_32_bits(fq):
    """Element offsets past 2^31 and byte offsets past 2^32: the last rows and columns of a long
    activation, and the last group's weights, against their own small calls."""
    rows, cols = 270000, 8192  # 2.2e9 elements
    x = torch.randn(rows // 1000, cols, device=DEV).to(torch.bfloat16).repeat(1000, 1)
    x[-300:] *= 3
    (q, d), (q_t, d_t) = fq.fp8_block_quant_dual(x)
    at = (rows - 300) // 128 * 128
    (q2, d2), (q_t2, d_t2) = fq.fp8_block_quant_dual(x[at:])
    assert torch.equal(q[at:], q2) and torch.equal(d[:, at:], d2)
    assert torch.equal(q_t[:, at:], q_t2) and torch.equal(d_t[at // 128:], d_t2)
    qr, dr = fq.fp8_block_quant_rowwise(x)
    assert torch.equal(qr[at:], q2) and torch.equal(dr, d)
    del x, qr, dr, q_t, d_t
    # the long operand's last rows, times the last of groups that lie past 4 GiB
    G, N = 70, 8192
    w = torch.randint(0, 120, (G, N, cols), dtype=torch.uint8, device=DEV)
    wd = torch.rand(G, N // 128, cols // 128, device=DEV)
    off = torch.full((G,), 0, dtype=torch.int32, device=DEV)
    off[-1] = rows - at
    y = fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q[at:], d[:, at:], w, wd, off)
    assert torch.equal(y, fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q2, d2, w[-1:].clone(), wd[-1:].clone()))


def test_outputs_past_the_last_level_cache(fq):
    """Outputs of more than 128 MiB, which are stored past the cache, hold the bits that the same rows and
    groups have in small calls; ragged in both directions."""
    M, N, K = 8195, 8200, 272
    q, d = fq.fp8_block_quant_rowwise(values(5, M, K))
    wq, _, wd = fq.fp8_block_quant_weights(values(6, N, K, 0.05), 1)
    b = wq.unflatten(0, (1, N))
    y = fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q, d, b, wd)
    for at in (0, 4096, 8192):
        rows = slice(at, min(at + 259, M))
        part = fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q[rows], d[:, rows].contiguous(), b, wd)
        assert torch.equal(y[rows], part)
    # weight gradient: 9 groups of 2808 x 2816, one without rows
    G, KK, NN, T = 9, 2808, 2816, 1100
    _, (a_t, a_s) = fq.fp8_block_quant_dual(values(7, T, KK))
    _, (g_t, g_s) = fq.fp8_block_quant_dual(values(8, T, NN))
    ends = [130, 256, 256, 300, 511, 700, 800, 1000, 1100]
    off = torch.tensor(ends, dtype=torch.int32, device=DEV)
    dw = fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, g_t, g_s, a_t, a_s, off)
    assert dw.shape[0] == G and dw.numel() * 2 > 128 << 20 and not bool(dw[2].any())
    for g in (0, 1, 3, 8):
        one = torch.tensor([ends[g - 1] if g else 0, ends[g]], dtype=torch.int32, device=DEV)
        part = fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, g_t, g_s, a_t, a_s, one)
        assert torch.equal(dw[g], part[1])


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,G,kind", [
    (200, 1000, 1040, 2, "cuts"), (1000, 1500, 400, 3, "cuts"), (130, 4100, 656, 1, "even"), (900, 1408, 2064, 4, "empties"),
    (1900, 1511, 272, 5, "cuts"), (700, 2048, 1168, 20, "empties"), (5000, 3500, 144, 6, "cuts"), (4700, 3600, 400, 5, "empties")])
def test_forward_by_tile(fq, M, N, K, G, kind, out):
    """Two sizes for each tile: 64 x 64, 128 x 64, 128 x 128 and 256 x 256."""
    test_forward(fq, M, N, K, G, kind, out)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,G,kind", [
    (1000, 500, 700, 1, "even"), (1333, 300, 260, 9, "empties"), (900, 700, 1030, 3, "cuts"), (700, 1500, 1300, 9, "cuts"),
    (400, 1530, 1290, 12, "empties")])
def test_weight_gradient_by_tile(fq, M, N, K, G, kind, out):
    """64-tiles (several steps ahead of the arithmetic, over groups' ends), 128- and 256-tiles."""
    test_weight_gradient(fq, M, N, K, G, kind, out)
