"""The few-token layer in 64 bits, with the bounds that it promises: 16 significant bits between the products,
sums in 32 bits, one rounding to bf16.  Test infrastructure only."""
from __future__ import annotations

import torch

from tests import blocklib as bl

U = 2.0 ** -24


def additions(blocks, parts, planes=1):
    """Additions that a sum goes through one after the other, at most: a block's 128 products (of each
    plane), the blocks of a part with their factors, the parts."""
    return 128 * planes + 2 * -(-blocks // parts) + parts + 2


def formula(x, ids, share, w13, s13, w2, s2, n1, n2, between=lambda h: h):
    """(y in 64 bits, how far sums of n1 and n2 additions, h in 16 bits and the join may be from it).
    between changes h, to plant a mistake."""
    T, H = x.shape
    E, I = w2.shape[0], w2.shape[2]
    x, share = x.cpu().double(), share.cpu().double()
    want, tol = torch.zeros(2, T, H, dtype=torch.float64).unbind(0)
    for e in sorted(set(ids.flatten().tolist())):
        if not 0 <= e < E:
            continue
        t, j = torch.nonzero(ids.cpu() == e, as_tuple=True)
        a, b = bl.real_square(w13[e], s13[e]), bl.real_square(w2[e], s2[e])
        gu, mags = x[t] @ a.t(), x[t].abs() @ a.abs().t()
        g, u, mg, mu = gu[:, :I], gu[:, I:], mags[:, :I], mags[:, I:]
        act = g * torch.sigmoid(g)
        h = act * u
        # |silu'| < 1.1; h's two planes leave half a step of the second, 2^-8 of at most 2^-8
        off = n1 * U * (1.1 * mg * u.abs() + act.abs() * mu) + 1.1 * (n1 * U) ** 2 * mg * mu + (2.0 ** -16 + 8 * U) * h.abs()
        b_abs, s = b.abs(), share[t, j][:, None]
        want.index_add_(0, t, s * (between(h) @ b.t()))
        tol.index_add_(0, t, s.abs() * (off @ b_abs.t() + (n2 + ids.shape[1] + 1) * U * ((h.abs() + off) @ b_abs.t())))
    return want, tol


def check(y, want, tol):
    off = (y.cpu().double() - want).abs()
    assert bool(torch.isfinite(off).all())
    assert float((off - tol * (1 + 2.0 ** -8) - 2.0 ** -8 * want.abs()).max()) <= 0
    # in the norm, what rounding the exact result to bf16 costs, and little more: h in one bf16 would
    # add as much again
    rounding = float((want.to(torch.bfloat16).double() - want).norm())
    assert float(off.norm()) <= 1.05 * rounding + 2.0 ** -12 * float(want.norm())
