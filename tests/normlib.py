"""The norm with 8-bit rows and its gradients in 64 bits, with bounds for sums, products and roots in 32 bits.
Test infrastructure only."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
GRID = {1: (448.0, -6, torch.float8_e4m3fn), 0: (240.0, -7, torch.float8_e4m3fnuz)}  # largest value, smallest exponent, type


def additions(cols):
    """Additions that a row's sum goes through one after the other, at most: a lane's, and the lanes' tree."""
    return cols // 64 + 16


def grid(v, fmt):
    """Nearest value of the 8-bit grid, ties to even, saturating."""
    top, emin, _ = GRID[fmt]
    v = v.clamp(-top, top)
    step = torch.exp2((torch.frexp(v)[1].double() - 1).clamp(min=emin) - 3)
    return torch.round(v / step) * step


def decode(q, fmt):
    return q.cpu().view(GRID[fmt][2]).double()


def stream(x, residual):
    """h: the sum of two bf16 values is rounded once to bf16 (64 bits hold it, 32 bits too where it matters)."""
    return x.cpu() if residual is None else (x.cpu().double() + residual.cpu().double()).to(torch.bfloat16)


def norm(h, w, eps):
    """(rstd, y, how far y in 32 bits may be from it, relative to it)."""
    h, w = h.cpu().double(), w.cpu().double()
    eps = float(np.float32(eps))  # the call takes it in 32 bits
    rstd = 1 / torch.sqrt(h.square().mean(1) + eps)
    # the sum of squares (a product and the additions), halved by the root; mean, eps, root and quotient; two products
    return rstd, h * rstd[:, None] * w, U * ((additions(h.shape[1]) + 1) / 2 + 6)


def check_norm(n, x, residual, w, eps, scaling, fmt, bf16):
    h = stream(x, residual)
    assert torch.equal(n.h.cpu().view(torch.int16), h.view(torch.int16))
    rstd, y, rel = norm(h, w, eps)
    assert bool(((n.rstd.cpu().double() - rstd).abs() <= rel * rstd).all())
    if bf16 or scaling is None:
        off = (n.y.cpu().double() - y).abs()
        # half a step, of a value that may have moved; subnormals of bf16 are 2^-133 apart
        assert bool((off <= (2.0 ** -8 * (1 + rel) + rel) * y.abs() + 2.0 ** -134).all())
    else:
        assert n.y is None
    if scaling is None:
        assert n.q is None and n.scales is None
        return
    top = GRID[fmt][0]
    width = x.shape[1] if scaling == "row" else 128
    at = torch.arange(x.shape[1]) // width
    amax = torch.zeros(x.shape[0], int(at[-1]) + 1, dtype=torch.float64).scatter_reduce(1, at.expand_as(y), y.abs(), "amax")
    s = top / amax.clamp(min=float(np.float32(1e-12)))
    got = n.scales.cpu().double()
    got = got[:, None] if scaling == "row" else 1 / got.t()
    assert got.shape == s.shape
    assert bool(((got - s).abs() <= (rel + 3 * U) * s).all())  # of amax; quotient, factor and its inverse here
    # rounding to the grid is monotonic: the byte lies between those of both ends of where y s may be.  The
    # product's own rounding below the normal range is under 2^-149.
    ys, slack = y * s[:, at], 2 * rel + 4 * U
    v = decode(n.q, fmt)
    ends = torch.stack([ys * (1 - slack), ys * (1 + slack)])
    assert bool((v >= grid(ends.amin(0) - 2.0 ** -140, fmt)).all()) and bool((v <= grid(ends.amax(0) + 2.0 ** -140, fmt)).all())
    assert bool(torch.isfinite(v).all())


def backward(dy, h, rstd, w, dh):
    """(dx, bound in 32 bits before its type's rounding, dw, its bound)."""
    dy, h, rstd, w = (t.cpu().double() for t in (dy, h, rstd, w))
    n, xh, g = h.shape[1], h * rstd[:, None], dy * w
    c = (g * xh).mean(1, keepdim=True)
    off_c = U * (additions(n) + 5) * (g * xh).abs().mean(1, keepdim=True)
    dx = rstd[:, None] * (g - xh * c)
    bound = rstd[:, None] * (4 * U * g.abs() + xh.abs() * (off_c + 5 * U * c.abs()))
    if dh is not None:
        dx = dx + dh.cpu().double()
        bound = bound + U * dx.abs()
    return dx, bound, (dy * xh).sum(0), U * (h.shape[0] + 8) * (dy * xh).abs().sum(0)


def check_backward(dx, dw, dy, h, rstd, w, dh):
    want, bound, want_w, bound_w = backward(dy, h, rstd, w, dh)
    half = torch.finfo(dx.dtype).eps / 2
    tiny = 2.0 ** -133  # below the normal range
    assert bool(((dx.cpu().double() - want).abs() <= (1 + half) * bound + half * want.abs() + tiny).all())
    assert bool(((dw.cpu().double() - want_w).abs() <= bound_w + tiny).all())
