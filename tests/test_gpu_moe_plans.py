"""The few-token layer on every path that its launches take, against 64 bits with the bounds that it
promises: 16 significant bits between the products, sums in 32 bits, one rounding to bf16."""
from __future__ import annotations

import pytest
import torch

from tests import block_cases, planlib
from tests import blocklib as bl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_quantization_grouped_amd as m
    m.lib()
    return m


def weights(g, E, n, k):
    """Random finite codes and factors that make rows of about unit size."""
    w = torch.randint(0, 256, (E, n, k), dtype=torch.uint8, device=DEV, generator=g)
    w[(w & 0x7F) == 0x7F] = 0x38
    up = lambda v: -(-v // 128)
    return w, (0.5 + torch.rand(E, up(n), up(k), device=DEV, generator=g)) / (120 * k ** 0.5)


def additions(blocks, parts, planes=1):
    """Additions that a sum goes through one after the other, at most: a block's 128 products (of each
    plane), the blocks of a part with their factors, the parts."""
    return 128 * planes + 2 * -(-blocks // parts) + parts + 2


def formula(x, ids, share, w13, s13, w2, s2, n1, n2):
    """(y in 64 bits, how far sums of n1 and n2 additions, h in 16 bits and the join may be from it)."""
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
        want.index_add_(0, t, s * (h @ b.t()))
        tol.index_add_(0, t, s.abs() * (off @ b_abs.t() + (n2 + ids.shape[1] + 1) * U * ((h.abs() + off) @ b_abs.t())))
    return want, tol


@pytest.mark.parametrize("name", list(block_cases.LAYERS))
def test_layer(fq, name):
    (T, k, E, H, I, few), gate_up, down = block_cases.LAYERS[name]
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert planlib.stream(False, T, k, E, H, I, cus) == gate_up and planlib.stream(True, T, k, E, H, I, cus) == down
    g = torch.Generator(device=DEV).manual_seed(T + H)
    w13, s13 = weights(g, E, 2 * I, H)
    w2, s2 = weights(g, E, H, I)
    x = torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16)
    # the experts in use are the last ones; most tokens share one, and one choice is of an expert elsewhere
    ids = torch.randint(E - few, E, (T, k), device=DEV, generator=g).to(torch.int32)
    ids[: T * 3 // 4, 0] = E - 1
    if k > 1:
        ids[T // 2, 1] = -1
    share = torch.rand(T, k, device=DEV, generator=g) + 0.25
    y = fq.fp8_moe_few_tokens(x, ids, share, w13, s13, w2, s2)
    want, tol = formula(x, ids, share, w13, s13, w2, s2, additions(-(-H // 128), gate_up[2]), additions(-(-I // 128), down[2], 2))
    off = (y.cpu().double() - want).abs()
    assert bool(torch.isfinite(off).all())
    assert float((off - tol * (1 + 2.0 ** -8) - 2.0 ** -8 * want.abs()).max()) <= 0
    # in the norm, what rounding the exact result to bf16 costs, and little more: h in one bf16 would
    # add as much again
    rounding = float((want.to(torch.bfloat16).double() - want).norm())
    assert float(off.norm()) <= 1.05 * rounding + 2.0 ** -12 * float(want.norm())
    assert torch.equal(y, fq.fp8_moe_few_tokens(x, ids, share, w13, s13, w2, s2))
