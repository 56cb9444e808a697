"""The plain gradient that the router's kernels are held to, against autograd and differences; and the calls'
refusals, without a GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

import fp8_quantization_grouped_amd as fq
from tests import routelib as rl
from tests.test_binding_cpu import BF16, calls, gpu, zeros  # noqa: F401


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_formula_is_the_derivative(scoring, renormalize):
    g = torch.Generator().manual_seed(1)
    T, E, k = 20, 7, 3
    l = torch.randn(T, E, generator=g, dtype=torch.float64)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    seq = torch.tensor([4, 4, 17])  # one empty, three tokens behind the last
    dw, dloss = torch.randn(T, k, generator=g), torch.randn(3, generator=g)

    def total(v):
        return (rl.balance(v, ids, scoring, seq)[0] * dloss).sum() + (rl.weights(v, ids, scoring, renormalize, 2.5) * dw).sum()

    v = l.clone().requires_grad_()
    total(v).backward()
    counts = rl.counts_of(ids, E, T, seq)
    want, bound = rl.gradient(l, ids, dw, scoring, renormalize, 2.5, dloss, counts, seq)
    assert float((v.grad - want).abs().max()) < 1e-12 and float(bound.max()) < 1e-3
    d = torch.randn(T, E, generator=g, dtype=torch.float64)
    diff = (total(l + 1e-5 * d) - total(l - 1e-5 * d)) / 2e-5
    assert abs(float(diff) - float((want * d).sum())) < 1e-8


P = ctypes.c_void_p(4096)  # never read
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def balance(**kw):
    a = dict(logits=P, dtype=1, T=4, E=8, ld=8, scoring=0, ids=P, k=2, seq=None, S=1, loss=P, counts=P, ws=P, size=1 << 20, stream=None)
    assert set(kw) <= set(a)
    return fq.lib().moe_balance(*{**a, **kw}.values())


def back(**kw):
    a = dict(logits=P, dtype=1, T=4, E=8, ld=8, scoring=0, ids=P, k=2, dw=P, renorm=1, scale=1.0, dloss=P, counts=P, seq=None, S=1,
             out=ctypes.c_void_p(8192), ld_d=8, stream=None)
    assert set(kw) <= set(a)
    return fq.lib().moe_route_backward(*{**a, **kw}.values())


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(ld=7), INVALID), (dict(k=0), INVALID), (dict(S=0), INVALID), (dict(S=2), INVALID),
    (dict(dtype=2), INVALID), (dict(scoring=2), INVALID), (dict(loss=None), INVALID), (dict(counts=None), INVALID),
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(ws=ctypes.c_void_p(4100)), INVALID), (dict(E=1025, ld=1025), UNSUPPORTED),
    (dict(k=33), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(T=1000, ws=None), WORKSPACE), (dict(T=1000, size=8), WORKSPACE)])
def test_balance_refuses(kw, status):
    assert balance(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(ld=7), INVALID), (dict(ld_d=7), INVALID), (dict(k=0), INVALID), (dict(S=0), INVALID),
    (dict(S=2), INVALID), (dict(counts=None), INVALID), (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(out=None), INVALID),
    (dict(out=P, ld_d=9), INVALID), (dict(dtype=-1), INVALID), (dict(scoring=3), INVALID), (dict(E=1025, ld=1025, ld_d=1025), UNSUPPORTED),
    (dict(k=33), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(T=0, logits=None, ids=None, out=None), OK)])
def test_backward_refuses(kw, status):
    assert back(**kw) == status


def test_routing_that_leaves_logits_refuses():
    f = fq.lib().moe_route_with_logits
    args = lambda ld: (P, 4, 64, 64, P, 8, 64, None, 0, 2, 1, 1.0, P, P, P, ld, P, 1 << 20, None)
    assert f(*args(7)) == INVALID


def test_binding_refuses(calls):  # noqa: F811
    l, ids, i32 = zeros(6, 8), zeros(6, 2, dtype=torch.int32), torch.int32
    for kw in (dict(logits=zeros(6, 8, dtype=torch.float16)), dict(logits=torch.zeros(6, 8)), dict(ids=zeros(6, 2)), dict(ids=zeros(5, 2, dtype=i32)),
               dict(ids=zeros(6, 4, dtype=i32)[:, ::2]), dict(scoring="tanh"), dict(sequences=zeros(2)), dict(sequences=zeros(1, 2, dtype=i32)),
               dict(loss=zeros(2)), dict(counts=zeros(1, 8)), dict(workspace=torch.zeros(64))):
        with pytest.raises(ValueError):
            fq.moe_balance(**{"logits": l, "ids": ids, **kw})
    counts, dloss = zeros(1, 8, dtype=i32), zeros(1)
    for kw in (dict(dweights=zeros(6, 3)), dict(dweights=zeros(6, 4)[:, ::2]), dict(dloss=None), dict(dloss=zeros(2)), dict(counts=None),
               dict(counts=zeros(2, 8, dtype=i32)), dict(dlogits=zeros(6, 8, dtype=BF16)), dict(dlogits=zeros(6, 7))):
        with pytest.raises(ValueError):
            fq.moe_route_backward(**{"logits": l, "ids": ids, "dloss": dloss, "counts": counts, **kw})
    with pytest.raises(ValueError, match="moe_route_backward"):
        fq.moe_balance(zeros(6, 8).requires_grad_(), ids)
    with pytest.raises(ValueError):
        fq.moe_route(zeros(4, 64, dtype=BF16), zeros(8, 64, dtype=BF16), 2, logits=zeros(4, 7))
    assert calls == []
