"""Renormalized routing weights where the chosen scores are tiny: they still are the scores over their
sum."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_quantization_grouped_amd as m
    m.lib()
    return m


def route(fq, logits, H, k, **kw):
    """Routing of one token per row of logits (bf16 values), each reached by one product."""
    T, E = logits.shape
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[range(T), range(T)] = 1
    r = torch.zeros(E, H, dtype=torch.bfloat16)
    r[:, :T] = logits.t()
    return fq.moe_route(x.to(DEV), r.to(DEV), k, **kw)


# one block per token, logits and choice apart, more than 256 experts
@pytest.mark.parametrize("H,E", [(16, 40), (2048, 64), (64, 300)])
@pytest.mark.parametrize("low", [-30, -50, -75, -87, -95, -110, -250, -3e4])
def test_sigmoids_of_very_negative_logits(fq, H, E, low):
    g = torch.Generator().manual_seed(E)
    logits = (low - 6 * torch.rand(5, E, generator=g)).to(torch.bfloat16)
    ids, w = route(fq, logits, H, 6, scoring="sigmoid", scale=2.5)
    l = torch.gather(logits.double(), 1, ids.cpu().long())
    # sigmoid(l) / sum of sigmoids, both times exp(-m)
    s = torch.exp(l - l.amax(1, keepdim=True)) / (1 + torch.exp(l))
    exact = 2.5 * s / s.sum(1, keepdim=True)
    # exponentials and quotients of a few units in the last place each, a sum of six
    assert bool(((w.cpu().double() - exact).abs() <= 2.0 ** -20 * exact + 2.0 ** -60).all())
    assert bool(((w.sum(1) - 2.5).abs() <= 2.5 * 2.0 ** -20).all())


@pytest.mark.parametrize("H,E", [(16, 40), (2048, 64), (64, 300)])
def test_a_bias_that_chooses_experts_of_vanishing_softmax(fq, H, E):
    logits = torch.zeros(4, E, dtype=torch.bfloat16)
    logits[:, 0] = torch.tensor([40.0, 75.0, 100.0, 300.0])
    logits[:, 5], logits[:, 9] = -1.0, 2.0
    bias = torch.zeros(E, device=DEV)
    bias[5], bias[9], bias[11] = 30, 20, 10
    ids, w = route(fq, logits, H, 3, bias=bias)
    assert ids.tolist() == [[5, 9, 11]] * 4
    exact = torch.softmax(torch.tensor([-1.0, 2.0, 0.0], dtype=torch.float64), 0)
    assert bool(((w.cpu().double() - exact).abs() <= 2.0 ** -20 * exact).all())


@pytest.mark.parametrize("H,E", [(16, 40), (2048, 64), (64, 300)])
def test_logits_of_minus_infinity(fq, H, E):
    """The token whose chosen logits are all minus infinity has no weight; one finite logit takes all."""
    x = torch.zeros(2, H, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1
    r = torch.zeros(E, H, dtype=torch.bfloat16, device=DEV)
    r[:, 0] = float("-inf")
    ids, w = fq.moe_route(x, r, 4, scoring="sigmoid")
    assert ids.tolist() == [[0, 1, 2, 3]] * 2 and not bool(w.any())
    r[7, 0] = -200
    ids, w = fq.moe_route(x, r, 4, scoring="sigmoid")
    assert ids.tolist() == [[7, 0, 1, 2]] * 2 and w.tolist() == [[1, 0, 0, 0]] * 2
