"""fp8_rms_norm and fp8_rms_norm_backward against 64 bits (tests/normlib.py)."""
from __future__ import annotations

import pytest
import torch

from tests import normlib as nl

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_quantization_grouped_amd as m
    m.lib()
    return m


def rows_of(rows, cols, seed, ld=None, shift=0, scale=1.0):
    """bf16 [rows, cols] with a few large columns; ld: elements between rows; shift: elements that the first one
    lies behind an allocation's start."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * scale
    x = torch.where(torch.rand(rows, cols, generator=g) < 0.01, x * 30, x).to(torch.bfloat16)
    ld = ld or cols
    flat = torch.full((rows * ld + shift,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = flat[shift:].view(rows, ld)[:, :cols]
    out.copy_(x)
    return out


def weight_of(cols, seed, dtype):
    return (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


SHAPES = [(1, 1), (1, 7), (2, 8), (3, 127), (5, 128), (4, 129), (700, 64), (130, 520), (1030, 1000), (1, 1024), (300, 2048),
          (33, 2064), (7, 1111), (65, 4096), (1, 7168), (40, 7168), (64, 8192), (17, 8200), (9, 16384), (2, 40000), (3, 32768)]
KINDS = [("block", 1, False), ("block", 1, True), ("row", 1, False), ("row", 0, True), (None, 1, True)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(fq, rows, cols, residual):
    x = rows_of(rows, cols, rows + cols)
    res = rows_of(rows, cols, 5 * rows + cols, scale=3.0) if residual else None
    for i, (scaling, fmt, bf16) in enumerate(KINDS):
        w = weight_of(cols, i, torch.float32 if i % 2 else torch.bfloat16)
        n = fq.fp8_rms_norm(x, w, EPS, residual=res, scaling=scaling, fmt=fmt, bf16=bf16)
        nl.check_norm(n, x, res, w, EPS, scaling, fmt, bf16)


@pytest.mark.parametrize("ld,shift", [(2064, 0), (2072, 8), (2065, 0), (2064, 1), (2064, 4)])
def test_norm_strides_and_alignments(fq, ld, shift):
    rows, cols = 37, 2056
    x, res = rows_of(rows, cols, 1, ld, shift), rows_of(rows, cols, 2, ld, shift)
    w = weight_of(cols + shift, 3, torch.bfloat16)[shift:]
    h, y = rows_of(rows, cols, 4, ld, shift), rows_of(rows, cols, 5, ld, shift)
    q = torch.zeros(rows, ld + 3, dtype=torch.uint8, device="cuda")[:, 3:cols + 3]
    s = torch.zeros(17, rows + 5, device="cuda")[:, :rows]
    n = fq.fp8_rms_norm(x, w, EPS, residual=res, h=h, y=y, q=q, scales=s)
    assert n.h is h and n.y is y and n.q is q and n.scales is s
    nl.check_norm(n, x, res, w, EPS, "block", 1, True)
    assert bool((h.as_strided((rows, ld - cols), (ld, 1), h.storage_offset() + cols) == 7).all())  # nothing between the rows
    assert bool((q._base[:, :3] == 0).all()) and bool((q._base[:, cols + 3:] == 0).all()) and bool((s._base[:, rows:] == 0).all())


@pytest.mark.parametrize("cols", [96, 2048, 1111])
def test_norm_of_extreme_rows(fq, cols):
    """Rows of zeros, of values whose squares vanish or overflow, and of one large value."""
    x = rows_of(6, cols, 1)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 2.0 ** 100
    x[3] = 3.0e38
    x[4] = 0
    x[4, cols // 2] = -2.5e38
    w = weight_of(cols, 2, torch.float32)
    for scaling, fmt, bf16 in KINDS:
        n = fq.fp8_rms_norm(x, w, EPS, scaling=scaling, fmt=fmt, bf16=bf16)
        nl.check_norm(n, x, None, w, EPS, scaling, fmt, bf16)


@pytest.mark.parametrize("rows,cols", [(9, 1000), (5, 77)])
def test_bytes_are_the_quantizers(fq, rows, cols):
    """Rows of one magnitude, a power of two, leave y = +-weight exactly: bytes and factors are those that the
    quantizers give those rows."""
    sign = torch.where(torch.rand(rows, cols, generator=torch.Generator().manual_seed(1)) < 0.5, -1.0, 1.0).cuda()
    x = (sign * torch.exp2(torch.arange(rows, device="cuda") - 3.0)[:, None]).to(torch.bfloat16)
    w = (torch.randn(cols, generator=torch.Generator().manual_seed(2)) * 3).to(torch.bfloat16).cuda()
    rows_y = (sign * w.float()).to(torch.bfloat16)
    n = fq.fp8_rms_norm(x, w, 1e-30, bf16=True)
    q, s = fq.fp8_block_quant_rowwise(rows_y)
    assert torch.equal(n.y, rows_y) and torch.equal(n.q, q) and torch.equal(n.scales, s)
    for fmt in (0, 1):
        n = fq.fp8_rms_norm(x, w, 1e-30, scaling="row", fmt=fmt)
        q, s = fq.fp8_quant_rowwise(rows_y, fmt)
        assert torch.equal(n.q, q) and torch.equal(n.scales, s)


@pytest.mark.parametrize("cols", [2048, 515])
def test_residual_in_place(fq, cols):
    for which in ("x", "residual"):
        x, res = rows_of(50, cols, 1), rows_of(50, cols, 2)
        w = weight_of(cols, 3, torch.bfloat16)
        want = fq.fp8_rms_norm(x, w, residual=res, bf16=True)
        got = fq.fp8_rms_norm(x, w, residual=res, bf16=True, h=x if which == "x" else res)
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_no_rows_and_no_columns(fq):
    w = weight_of(64, 1, torch.float32)
    n = fq.fp8_rms_norm(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), w)
    assert n.q.shape == (0, 64) and n.scales.shape == (1, 0)
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    dx, dw = fq.fp8_rms_norm_backward(empty, empty, torch.empty(0, device="cuda"), w)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and dw.shape == (64,)
    n = fq.fp8_rms_norm(torch.empty(3, 0, dtype=torch.bfloat16, device="cuda"), w[:0], scaling=None)
    assert n.y.shape == (3, 0)


# ------------------------------------------------------------------------------------ gradients

@pytest.mark.parametrize("rows,cols", SHAPES + [(2000, 64), (5000, 1000), (513, 2048), (1025, 257)])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_norm_backward(fq, rows, cols, grad):
    for with_dh in (False, True):
        h = rows_of(rows, cols, rows)
        w = weight_of(cols, 1, torch.bfloat16 if with_dh else torch.float32)
        rstd = fq.fp8_rms_norm(h, w, EPS, scaling=None).rstd
        dy = rows_of(rows, cols, rows + 1).to(grad)
        dh = rows_of(rows, cols, rows + 2).to(grad) if with_dh else None
        dx, dw = fq.fp8_rms_norm_backward(dy, h, rstd, w, dh=dh)
        assert dx.dtype == grad
        nl.check_backward(dx, dw, dy, h, rstd, w, dh)


@pytest.mark.parametrize("ld,shift", [(2072, 8), (2065, 0), (2064, 3)])
def test_norm_backward_strides_and_in_place(fq, ld, shift):
    rows, cols = 37, 2056
    h, dy, dh = (rows_of(rows, cols, i, ld, shift) for i in range(3))
    w = weight_of(cols, 3, torch.float32)
    rstd = fq.fp8_rms_norm(h, w, EPS, scaling=None).rstd
    want = fq.fp8_rms_norm_backward(dy, h, rstd, w, dh=dh, dx=rows_of(rows, cols, 9, ld, shift))
    nl.check_backward(*want, dy, h, rstd, w, dh)
    for into in (dy, dh):
        keep = into.clone()
        got, dw = fq.fp8_rms_norm_backward(dy, h, rstd, w, dh=dh, dx=into)
        assert got is into and torch.equal(got, want[0]) and torch.equal(dw, want[1])
        assert bool((into.as_strided((rows, ld - cols), (ld, 1), into.storage_offset() + cols) == 7).all())
        into.copy_(keep)


def test_norm_backward_repeats_to_the_bit(fq):
    h, dy = rows_of(3000, 1024, 1), rows_of(3000, 1024, 2)
    w = weight_of(1024, 3, torch.bfloat16)
    rstd = fq.fp8_rms_norm(h, w, scaling=None).rstd
    first = fq.fp8_rms_norm_backward(dy, h, rstd, w)
    for _ in range(3):
        for a, b in zip(first, fq.fp8_rms_norm_backward(dy, h, rstd, w)):
            assert torch.equal(a, b)


def test_norm_backward_against_differences(fq):
    """The forward in 64 bits at both sides of a step along a direction."""
    rows, cols = 6, 200
    h, dy = rows_of(rows, cols, 1), rows_of(rows, cols, 2).float()
    w = weight_of(cols, 3, torch.float32)
    rstd = fq.fp8_rms_norm(h, w, EPS, scaling=None).rstd
    dx, dw = fq.fp8_rms_norm_backward(dy, h, rstd, w)
    f = lambda a, b: float((nl.norm(a, b, EPS)[1] * dy.cpu().double()).sum())
    g = torch.Generator().manual_seed(4)
    v, u = torch.randn(rows, cols, generator=g, dtype=torch.float64), torch.randn(cols, generator=g, dtype=torch.float64)
    hd, wd, step = h.cpu().double(), w.cpu().double(), 1e-5
    diff = (f(hd + step * v, wd + step * u) - f(hd - step * v, wd - step * u)) / (2 * step)
    slope = float((dx.cpu().double() * v).sum() + (dw.cpu().double() * u).sum())
    _, b, _, bw = nl.backward(dy, h, rstd, w, None)
    # rstd in 32 bits enters to the third power; the differences' own error is of the order step^2
    size = float((dx.cpu().double().abs() * v.abs()).sum() + (dw.cpu().double().abs() * u.abs()).sum())
    slack = float((b * v.abs()).sum() + (bw * u.abs()).sum()) + 3 * nl.norm(h, w, EPS)[2] * 2 * size + 1e-7 * size
    assert abs(diff - slope) <= slack
