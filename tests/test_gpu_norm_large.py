"""The norm and its gradients at sizes past the last-level cache, where reads and writes go past the caches, and
on rows of every shape that registers hold: the same bits as in smaller pieces, which take the other accesses."""
from __future__ import annotations

import pytest
import torch

from tests import normlib as nl
from tests.test_gpu_norm import KINDS, fq, rows_of, weight_of  # noqa: F401

pytestmark = pytest.mark.gpu


def big(rows, cols, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("rows,cols", [(6000, 7168), (6001, 7165), (40000, 1000), (700000, 64), (2500, 16000), (1300, 32768), (20000, 2048)])
def test_norm_past_the_caches(fq, rows, cols):  # noqa: F811
    x, res, w = big(rows, cols, 1), big(rows, cols, 2), weight_of(cols, 3, torch.bfloat16)
    for scaling, fmt, bf16 in KINDS:
        whole = fq.fp8_rms_norm(x, w, residual=res, scaling=scaling, fmt=fmt, bf16=bf16)
        step = rows // 7 + 1  # more than 512 rows of up to 8192: fewer take another shape, whose sums have another order
        for at in range(0, rows, step):
            part = fq.fp8_rms_norm(x[at:at + step], w, residual=res[at:at + step], scaling=scaling, fmt=fmt, bf16=bf16)
            for name in ("h", "y", "q", "rstd"):
                a, b = getattr(whole, name), getattr(part, name)
                assert (a is None) == (b is None) and (a is None or torch.equal(a[at:at + step], b)), (name, at)
            if scaling:
                s = whole.scales[at:at + step] if scaling == "row" else whole.scales[:, at:at + step]
                assert torch.equal(s, part.scales)
    at = rows - 20
    end = fq.fp8_rms_norm(x[at:], w, residual=res[at:])
    nl.check_norm(end, x[at:], res[at:], w, 1e-6, "block", 1, False)


@pytest.mark.parametrize("rows,cols", [(6000, 7168), (6001, 7165), (40000, 1000), (700000, 64), (2500, 16000)])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_backward_past_the_caches(fq, rows, cols, grad):  # noqa: F811
    h, w = big(rows, cols, 1), weight_of(cols, 3, torch.float32)
    dy, dh = big(rows, cols, 2).to(grad), big(rows, cols, 4).to(grad)
    rstd = fq.fp8_rms_norm(h, w, scaling=None).rstd
    dx, dw = fq.fp8_rms_norm_backward(dy, h, rstd, w, dh=dh)
    step = rows // 7 + 1  # more than 512 rows of up to 8192: fewer take another shape, whose sums have another order
    for at in range(0, rows, step):
        part, _ = fq.fp8_rms_norm_backward(dy[at:at + step], h[at:at + step], rstd[at:at + step], w, dh=dh[at:at + step])
        assert torch.equal(dx[at:at + step], part), at
    terms = dy.double() * (h.double() * rstd.double()[:, None])
    assert bool(((dw.double() - terms.sum(0)).abs() <= nl.U * (rows + 8) * terms.abs().sum(0)).all())
    at = rows - 20
    nl.check_backward(dx[at:], fq.fp8_rms_norm_backward(dy[at:], h[at:], rstd[at:], w, dh=dh[at:])[1], dy[at:], h[at:], rstd[at:], w, dh[at:])


@pytest.mark.parametrize("cols", [300, 800, 1500, 3500, 4096, 7168, 12000, 20000])
def test_one_extreme_row_among_others(fq, cols):  # noqa: F811
    """Rows whose squares overflow beside rows whose do not, in one block and on every shape."""
    rows = 600
    x = rows_of(rows, cols, 1)
    for at in (0, 3, 5, 300, rows - 1):
        x[at] = 3.0e38 if at % 2 else 1.5e30
    w = weight_of(cols, 2, torch.float32)
    for scaling, fmt, bf16 in KINDS:
        for part in (x, x[:7]):
            n = fq.fp8_rms_norm(part, w, scaling=scaling, fmt=fmt, bf16=bf16)
            nl.check_norm(n, part, None, w, 1e-6, scaling, fmt, bf16)


def test_offsets_past_32_bits(fq):  # noqa: F811
    """Rows that lie more than 2^31 elements behind the first one."""
    rows, cols, ld = 5, 256, (1 << 31) // 4 + 40
    flat = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = flat.view(rows, ld)[:, :cols]
    x.copy_(rows_of(rows, cols, 1))
    w = weight_of(cols, 2, torch.float32)
    out = torch.empty(rows * ld, dtype=torch.uint8, device="cuda").view(rows, ld)[:, :cols]
    n = fq.fp8_rms_norm(x, w, q=out, bf16=True)
    nl.check_norm(n, x, None, w, 1e-6, "block", 1, True)
    dx, dw = fq.fp8_rms_norm_backward(x, x, n.rstd, w, dx=x.clone())
    nl.check_backward(dx, dw, x, x, n.rstd, w, None)
    got, _ = fq.fp8_rms_norm_backward(x, x.contiguous(), n.rstd, w, dx=x)
    assert torch.equal(got, dx)
