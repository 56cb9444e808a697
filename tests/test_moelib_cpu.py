"""The layer's 64-bit comparison takes a result of 16 bits between the products and refuses one of 8 (CPU)."""
from __future__ import annotations

import pytest
import torch

from tests import moelib


def one_plane(h):
    return h.to(torch.bfloat16).double()


def two_planes(h):
    return one_plane(h) + one_plane(h - one_plane(h))


@pytest.mark.parametrize("T,H,I,E,k", [(3, 256, 160, 4, 2), (40, 128, 384, 3, 2)])
def test_one_plane_is_found(T, H, I, E, k):
    g = torch.Generator().manual_seed(T)
    up = lambda n: -(-n // 128)

    def weights(n, m):
        w = torch.randint(0, 256, (E, n, m), dtype=torch.uint8, generator=g)
        w[(w & 0x7F) == 0x7F] = 0x38
        return w, (0.5 + torch.rand(E, up(n), up(m), generator=g)) / (120 * m ** 0.5)

    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    ids = torch.randint(0, E, (T, k), generator=g).to(torch.int32)
    args = (x, ids, torch.rand(T, k, generator=g) + 0.25, *weights(2 * I, H), *weights(H, I))
    n = moelib.additions(up(H), 1), moelib.additions(up(I), 1, 2)
    want, tol = moelib.formula(*args, *n)
    moelib.check(want.to(torch.bfloat16), want, tol)
    good, _ = moelib.formula(*args, *n, between=two_planes)
    moelib.check(good.to(torch.bfloat16), want, tol)
    bad, _ = moelib.formula(*args, *n, between=one_plane)
    with pytest.raises(AssertionError):
        moelib.check(bad.to(torch.bfloat16), want, tol)
