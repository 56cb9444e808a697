"""Refusals of AdamWStates and adamw_step and what they hand on, without a GPU; and the rounding's random bits."""
from __future__ import annotations

import ctypes

import pytest
import torch

import fp8_quantization_grouped_amd as fq
from tests import adamlib as al
from tests.test_binding_cpu import BF16, U8, calls, gpu, zeros  # noqa: F401

OK, INVALID, UNSUPPORTED = 0, 1, 2


def step(tensor={}, count=1, **kw):
    t = fq._AdamTensor(**{**dict(param=4096, grad=8192, exp_avg=4096 * 3, exp_avg_scales=4096 * 4, exp_avg_sq=4096 * 5,
                                 exp_avg_sq_scales=4096 * 6, n=4, param_dtype=0, grad_dtype=0), **tensor})
    h = fq._Adam(**{**dict(beta1=0.9, beta2=0.99, step=1, lr=1e-3, eps=1e-8, weight_decay=0.0, state_bits=8), **kw})
    return fq.lib().adamw_step(ctypes.addressof(t), count, ctypes.addressof(h), None)


@pytest.mark.parametrize("kw", [
    dict(count=-1), dict(state_bits=16), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=float("nan")), dict(eps=0.0), dict(eps=-1.0),
    dict(step=0), dict(step=-3), dict(tensor=dict(n=-1)), dict(tensor=dict(param_dtype=2)), dict(tensor=dict(grad_dtype=-1)),
    dict(tensor=dict(param=None)), dict(tensor=dict(exp_avg=None)), dict(tensor=dict(exp_avg_sq=None)), dict(tensor=dict(exp_avg_scales=None)),
    dict(tensor=dict(exp_avg_sq_scales=None)), dict(tensor=dict(master=4096, param_dtype=1))])
def test_step_refuses(kw):
    assert step(**kw) == INVALID


def test_step_limits_and_nothing_to_do():
    assert step(tensor=dict(n=(1 << 34) + 1)) == UNSUPPORTED
    assert step(count=0) == OK and step(tensor=dict(n=0, param=None)) == OK and step(tensor=dict(grad=None, param=None)) == OK
    assert fq.lib().adamw_step(None, 1, None, None) == INVALID


def states(params, masters=None):
    """8-bit states on tensors of the host that the binding takes for a GPU's."""
    many = lambda dtype, size: [zeros(size(p.numel()), dtype=dtype) for p in params]
    whole, blocks = lambda n: n, lambda n: -(-n // 128)
    return fq.AdamWStates(params, 8, masters, many(U8, whole), many(U8, whole), many(torch.float32, blocks), many(torch.float32, blocks))


def test_states_of_memory_that_overlaps(calls):  # noqa: F811
    all_ = zeros(300)
    for params in ([all_[:200], all_[100:]], [all_, all_[299:]], [all_[10:20], all_[:300]]):
        with pytest.raises(ValueError, match="share memory"):
            states(params)
    states([all_[:100], all_[100:300]])


def test_step_refuses_parameters_of_other_memory(calls):  # noqa: F811
    for other in (lambda p: zeros(4, 4), lambda p: p.data.t(), lambda p: p.data[:2]):
        p = zeros(4, 4)
        s = states([p])
        fq.adamw_step(s, [zeros(4, 4)], 1, 1e-3)
        p.data = other(p)
        with pytest.raises(ValueError, match="other memory"):
            fq.adamw_step(s, [zeros(*p.shape)], 2, 1e-3)
        fq.adamw_step(s, [None], 2, 1e-3)
    p, m = zeros(4, 4, dtype=BF16), zeros(4, 4)
    s = states([p], [m])
    m.data = zeros(4, 4)
    with pytest.raises(ValueError, match="other memory"):
        fq.adamw_step(s, [zeros(4, 4)], 1, 1e-3)
    assert len(calls) == 6


def test_step_tells_torch_of_what_it_changes_alone(calls):  # noqa: F811
    p, m = [zeros(8, dtype=BF16), zeros(8)], [zeros(8), None]
    s = states(p, m)
    before = [t._version for t in (p[0], m[0], p[1])]
    fq.adamw_step(s, [None, zeros(8)], 1, 1e-3)
    assert [t._version for t in (p[0], m[0], p[1])] == [before[0], before[1], before[2] + 1]
    fq.adamw_step(s, [zeros(8), None], 2, 1e-3)
    assert [t._version for t in (p[0], m[0], p[1])] == [before[0] + 1, before[1] + 1, before[2] + 1]


def test_states_refuse(calls):  # noqa: F811
    p = [zeros(4, 8), zeros(300, dtype=BF16)]
    same = zeros(32)
    m8 = lambda: [zeros(32, dtype=U8), zeros(300, dtype=U8)]
    f8 = lambda: [zeros(1), zeros(3)]
    for args, kw in (((p, 16), {}), (([zeros(4, dtype=torch.float16)],), {}), (([torch.zeros(4)],), {}), (([zeros(4, 8).t()],), {}),
                     ((p,), dict(masters=[None])), ((p,), dict(masters=[zeros(4, 8), None])), ((p,), dict(masters=[None, zeros(300, dtype=BF16)])),
                     ((p,), dict(masters=[None, zeros(299)])), ((p,), dict(exp_avg=m8())), ((p,), dict(exp_avg=m8(), exp_avg_sq=m8())),
                     ((p, 32), dict(exp_avg=m8(), exp_avg_sq=m8())), ((p, 32), dict(exp_avg_scales=f8())),
                     ((p,), dict(exp_avg=m8(), exp_avg_sq=m8(), exp_avg_scales=f8(), exp_avg_sq_scales=[zeros(1), zeros(2)])),
                     (([same, same],), {}), ((p[:1], 32), dict(exp_avg=[same], exp_avg_sq=[same]))):
        with pytest.raises(ValueError):
            fq.AdamWStates(*args, **kw)
    assert calls == []


def test_step_binding_refuses(calls):  # noqa: F811
    s = states([zeros(4, 8)])
    g = [zeros(4, 8)]
    for kw in (dict(grads=[]), dict(grads=[zeros(32)]), dict(grads=[zeros(4, 8, dtype=torch.float16)]), dict(grads=[torch.zeros(4, 8)]),
               dict(grads=[zeros(8, 4).t()]), dict(step=0), dict(step=zeros(1)), dict(step=zeros(2, dtype=torch.int32)),
               dict(lr=zeros(1, dtype=BF16)), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -1.0)), dict(eps=0.0), dict(grad_scale=0.5),
               dict(grad_scale=zeros(2)), dict(step=torch.ones(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            fq.adamw_step(s, **{"grads": g, "step": 1, "lr": 1e-3, **kw})
    assert calls == []
    fq.adamw_step(s, g, 3, 1e-3)
    fq.adamw_step(s, [None], zeros(1, dtype=torch.int32), zeros(1), grad_scale=zeros(1))
    assert len(calls) == 2


def test_the_random_bits_are_even():
    """Each of the 32 bits, and the upper 20 of the word and of its halves exchanged as numbers, over a tensor,
    over tensors and over steps."""
    runs = [al.words(1, 0, 1 << 16), torch.stack([al.words(s, 0, 16) for s in range(4096)]).flatten(),
            torch.stack([al.words(7, i, 16) for i in range(4096)]).flatten()]
    for w in runs:
        n = len(w)
        for b in range(32):
            assert abs(float(((w >> b) & 1).double().mean()) - 0.5) < 6 * 0.5 / n ** 0.5
        for v in (w, ((w << 16) | (w >> 16)) & 0xFFFFFFFF):
            u = (v >> 12).double() / 2 ** 20
            assert abs(float(u.mean()) - 0.5) < 6 * 0.29 / n ** 0.5
            counts = torch.histc(u, 64, 0, 1)
            assert float(((counts - n / 64) ** 2 / (n / 64)).sum()) < 63 + 6 * (2 * 63) ** 0.5  # chi-square
        both = torch.corrcoef(torch.stack([(w >> 12).double(), ((((w << 16) | (w >> 16)) & 0xFFFFFFFF) >> 12).double()]))[0, 1]
        assert abs(float(both)) < 6 / n ** 0.5 + 2.0 ** -10
        assert abs(float(torch.corrcoef(torch.stack([w[:-1].double(), w[1:].double()]))[0, 1])) < 6 / n ** 0.5
