"""The weight's gradient of the norm by whole numbers: h, rstd and dy are powers of two and small whole numbers, so
that every product and every sum of them is exact in 32 bits, in any order, and a row that is lost or added twice
by any block shows.  (A bound for rounded sums grows with the rows, past what one block of many brings.)"""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_norm import SHAPES, fq, weight_of  # noqa: F401

pytestmark = pytest.mark.gpu


def whole(rows, cols, seed, grad):
    """h, rstd, dy and the sums over rows of dy h rstd: terms are multiples of 1/4 up to 16, and the sums of up to
    2^18 rows stay under 2^24 quarters; more rows take terms up to 1."""
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device="cuda")
    small = rows > 1 << 18
    h = (torch.exp2(r(-1, 1 if small else 2, rows, cols).float()) * (1 - 2 * r(0, 2, rows, cols))).to(torch.bfloat16)
    rstd = torch.exp2(r(-1, 1 if small else 2, rows).float())
    dy = r(-1, 2, rows, cols) if small else r(-4, 5, rows, cols)
    dy = dy.to(grad)
    want = torch.zeros(cols, dtype=torch.float64, device="cuda")
    for at in range(0, rows, 1 << 14):
        part = slice(at, at + (1 << 14))
        want += (dy[part].double() * h[part].double() * rstd[part].double()[:, None]).sum(0)
    return h, rstd, dy, want


MANY = [(255, 64), (256, 64), (4097, 64), (4096, 512), (5000, 513), (3000, 1024), (1537, 2064), (2000, 4104), (777, 7168), (600, 8192), (513, 8200),
        (300, 16384), (257, 16392), (300, 7), (6001, 7165), (40000, 1000), (700000, 64), (2500, 16000)]


@pytest.mark.parametrize("rows,cols", SHAPES + MANY)
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_every_row_counts_once(fq, rows, cols, grad):  # noqa: F811
    h, rstd, dy, want = whole(rows, cols, rows + cols, grad)
    assert float(want.abs().max()) < 1 << 22
    w = weight_of(cols, 1, torch.bfloat16 if rows % 2 else torch.float32)
    _, dw = fq.fp8_rms_norm_backward(dy, h, rstd, w)
    assert torch.equal(dw.double(), want)


@pytest.mark.parametrize("ld,shift", [(2072, 8), (2065, 0), (2064, 3)])
def test_every_row_counts_once_at_any_stride(fq, ld, shift):  # noqa: F811
    rows, cols = 1000, 2056
    h, rstd, dy, want = whole(rows, cols, ld, torch.bfloat16)

    def spaced(t):
        out = torch.full((rows * ld + shift,), 7.0, dtype=t.dtype, device="cuda")[shift:].view(rows, ld)[:, :cols]
        return out.copy_(t)

    _, dw = fq.fp8_rms_norm_backward(spaced(dy), spaced(h), rstd, weight_of(cols, 1, torch.float32), dh=spaced(h))
    assert torch.equal(dw.double(), want)
