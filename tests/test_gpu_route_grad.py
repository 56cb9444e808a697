"""moe_balance, moe_route_backward and the logits that moe_route leaves, against 64 bits (tests/routelib.py)."""
from __future__ import annotations

import pytest
import torch

from tests import routelib as rl

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_quantization_grouped_amd as m
    m.lib()
    return m


def case(T, E, k, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    l = (torch.randn(T, E, generator=g) * 2).to(dtype).cuda()
    ids = torch.argsort(torch.rand(T, E, generator=g), 1)[:, :k].to(I32).contiguous().cuda()
    return l, ids, torch.randn(T, k, generator=g).cuda()


def run(fq, l, ids, dw, scoring="softmax", renormalize=True, scale=1.0, sequences=None, balance=True):
    """Both calls and their checks."""
    loss, counts = fq.moe_balance(l, ids, scoring=scoring, sequences=sequences)
    rl.check_balance(loss, counts, l, ids, scoring, sequences)
    dloss = torch.linspace(0.5, 1.5, loss.shape[0]).cuda() if balance else None
    on = dict(dloss=dloss, counts=counts, sequences=sequences) if balance else {}
    d = fq.moe_route_backward(l, ids, dw, scoring=scoring, renormalize=renormalize, scale=scale, **on)
    assert d.dtype == l.dtype
    rl.check_gradient(d, l, ids, dw, scoring, renormalize, scale, dloss, counts, sequences)
    return loss, counts, d


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (3, 1), (4, 2), (5, 5), (8, 2), (13, 3), (16, 4), (31, 2), (32, 8), (64, 6), (65, 7), (100, 1),
                                 (128, 8), (200, 32), (256, 8), (300, 9), (512, 16), (777, 3), (1024, 8)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_numbers_of_experts(fq, E, k, scoring):
    for i, T in enumerate((1, 67, 500)):
        l, ids, dw = case(T, E, k, E + T, torch.bfloat16 if i == 1 else torch.float32)
        for renormalize in (True, False):
            run(fq, l, ids, dw, scoring, renormalize, scale=1.0 if renormalize else 2.5)


@pytest.mark.parametrize("T,ends", [
    (1, [1]), (7, [0, 7]), (100, [40, 40, 40, 41, 100]), (100, [3, 10, 60]), (1000, [999]), (1000, list(range(1, 1001))),
    (4096, [1, 4000, 4096]), (5000, [0] * 300 + [2500] * 2 + [4990]), (9000, [9000]), (33, [0, 0]), (600, list(range(3, 600, 7)))])
def test_sequences(fq, T, ends):
    for E, k in ((8, 2), (64, 6), (260, 4)):
        l, ids, dw = case(T, E, k, T + E)
        run(fq, l, ids, dw, sequences=torch.tensor(ends, dtype=I32).cuda())


def test_tokens_behind_the_last_sequence_have_the_weights_gradient_alone(fq):
    l, ids, dw = case(50, 16, 2, 1)
    _, counts, d = run(fq, l, ids, None, sequences=torch.tensor([30], dtype=I32).cuda())
    assert bool((d[30:] == 0).all()) and int(counts.sum()) == 60
    _, _, d = run(fq, l, ids, dw, sequences=torch.tensor([30], dtype=I32).cuda())
    assert torch.equal(d[30:], run(fq, l, ids, dw, balance=False)[2][30:])


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_and_extreme_logits(fq, scoring, dtype):
    l, ids, dw = case(64, 40, 4, 3, dtype)
    inf = float("inf")
    l[0:8, 5:] = -inf              # most experts masked out
    l[8:16] = -inf                 # all of them: no probabilities, no gradients
    l[16:24, 1:] = torch.finfo(dtype).min
    l[24:32] = l[24:32] - 200      # sigmoids that vanish
    l[32:40] = l[32:40] * 1000
    l[40:48, ::2] = -90
    l[48:50] = torch.finfo(dtype).min
    l[50:52] = 0
    ids[56:58] = -1                # a padded token's choices
    ids[58:60] = 40
    ids[60:62] = ids[60:62, :1]    # the same expert every time
    ids[62:64, 2:] = ids[62:64, :2]
    for renormalize in (True, False):
        _, _, d = run(fq, l, ids, dw, scoring, renormalize)
        assert bool(torch.isfinite(d).all()) and bool((d[8:16] == 0).all())


def test_chosen_logits_far_below_the_others(fq):
    """A bias can choose experts whose scores vanish beside the rest: their weights are ratios all the same."""
    l, ids, dw = case(32, 24, 3, 5)
    far = torch.zeros(32, 24).scatter_(1, ids.cpu().long(), -100.0).cuda()
    for scoring in ("softmax", "sigmoid"):
        run(fq, l + far, ids, dw, scoring, balance=False)


@pytest.mark.parametrize("ld,shift", [(64, 0), (68, 4), (67, 0), (64, 1), (66, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_in_place(fq, ld, shift, dtype):
    T, E, k = 77, 60, 4
    base, ids, dw = case(T, E, k, 9, dtype)
    flat = torch.full((T * ld + shift,), 7.0, dtype=dtype, device="cuda")
    l = flat[shift:].view(T, ld)[:, :E]
    l.copy_(base)
    want = run(fq, l, ids, dw)[2]
    assert torch.equal(want, run(fq, base, ids, dw)[2])
    loss, counts = fq.moe_balance(l, ids)
    got = fq.moe_route_backward(l, ids, dw, dloss=torch.ones(1, device="cuda") * 0.5, counts=counts, dlogits=l)
    assert got is l and torch.equal(l, want)
    assert bool((flat[shift:].view(T, ld)[:, E:] == 7).all()) and bool((flat[:shift] == 7).all())


def test_no_tokens(fq):
    l, ids = torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=I32, device="cuda")
    for seq, S in ((None, 1), (torch.zeros(3, dtype=I32, device="cuda"), 3)):
        loss, counts = fq.moe_balance(l, ids, sequences=seq)
        assert loss.shape == (S,) and bool((loss == 0).all()) and counts.shape == (S, 8) and bool((counts == 0).all())
    assert fq.moe_route_backward(l, ids, torch.empty(0, 2, device="cuda")).shape == (0, 8)


def test_any_ends_stay_inside(fq):
    """Ends that do not grow, or lie outside: results are unspecified, accesses are not."""
    l, ids, dw = case(3000, 64, 2, 1)
    for ends in ([2000, 100, 3000], [-5, 1 << 30, 7], [1 << 30] * 4, [-1, -1]):
        seq = torch.tensor(ends, dtype=I32).cuda()
        _, counts = fq.moe_balance(l, ids, sequences=seq)
        fq.moe_route_backward(l, ids, dw, dloss=torch.ones(len(ends), device="cuda"), counts=counts, sequences=seq)
    torch.cuda.synchronize()


def test_results_repeat_to_the_bit(fq):
    l, ids, dw = case(20000, 96, 6, 2)
    first = run(fq, l, ids, dw)
    for _ in range(3):
        for a, b in zip(first, run(fq, l, ids, dw)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,H,E,k", [(3, 64, 4, 2), (40, 256, 64, 6), (200, 2048, 64, 6), (17, 512, 300, 8), (5, 1024, 1000, 4)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_logits_of_the_routing(fq, T, H, E, k, scoring):
    """moe_route's logits on each of its paths: its ids and weights as without them, the logits x Wr^T, and the
    weights that they give are the returned ones."""
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    router = (torch.randn(E, H, generator=g) * H ** -0.5).to(torch.bfloat16).cuda()
    bias = torch.randn(E, generator=g).cuda() * 0.1
    ids, w = fq.moe_route(x, router, k, bias=bias, scoring=scoring)
    wide = torch.full((T, E + 3), 7.0, device="cuda")
    ids2, w2 = fq.moe_route(x, router, k, bias=bias, scoring=scoring, logits=wide[:, :E])
    assert torch.equal(ids, ids2) and torch.equal(w, w2) and bool((wide[:, E:] == 7).all())
    l = wide[:, :E].contiguous()
    exact, mags = x.cpu().double() @ router.cpu().double().t(), x.cpu().double().abs() @ router.cpu().double().abs().t()
    assert bool(((l.cpu().double() - exact).abs() <= H * rl.U * mags).all())
    got = rl.weights(l.cpu().double(), ids, scoring, True, 1.0)
    # scores, their sum and the quotient in 32 bits, exponents up to 20 away
    assert bool(((w.cpu().double() - got).abs() <= (2 * (20 + 8) + 64) * rl.U * got).all())
    run(fq, l, ids, torch.randn(T, k, generator=g).cuda(), scoring)


@pytest.mark.parametrize("E,k", [(4, 2), (16, 3), (64, 6), (256, 8), (1000, 4)])
def test_one_block_or_more(fq, E, k):
    """As many tokens as one block takes by itself, and one more; with and without sequences, empty ones first, in
    the middle and last."""
    once = 512
    while 16 * 512 // once < E:
        once //= 2
    assert fq.moe_balance_workspace_size(once, E, 1) == 0 < fq.moe_balance_workspace_size(once + 1, E, 1)
    for T in (once - 1, once, once + 1):
        l, ids, dw = case(T, E, k, T)
        run(fq, l, ids, dw)
        for ends in ([0, 0, 1, T // 2, T // 2, T - 1, T - 1], [T], [0] * 70 + [T]):
            run(fq, l, ids, dw, sequences=torch.tensor(ends, dtype=I32).cuda())


@pytest.mark.parametrize("T,E,k,ends", [(30000, 512, 4, [10, 29000]), (20000, 1000, 2, None), (40000, 257, 8, [0, 39999, 39999, 40000]), (9000, 260, 3, [8999])])
def test_joins_in_groups_of_experts(fq, T, E, k, ends):
    """Sums of a sequence that several blocks join."""
    l, ids, dw = case(T, E, k, T)
    seq = None if ends is None else torch.tensor(ends, dtype=I32).cuda()
    first = run(fq, l, ids, dw, sequences=seq)
    for a, b in zip(first, run(fq, l, ids, dw, sequences=seq)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,E,k", [(300, 8, 2), (5000, 64, 6)])
def test_many_empty_sequences(fq, T, E, k):
    """Runs of empty sequences before, between and behind tokens' ones: the losses and counts of those with tokens
    as without the empty ones, zeros for these, and the same gradient to the bit."""
    l, ids, dw = case(T, E, k, T)
    ends, few = [], [T // 3, T // 3 + 1, T - 7]
    at = []
    for before, e in zip([0] + few, few):
        ends += [before] * 30011 + [e]
        at.append(len(ends) - 1)
    ends = torch.tensor(ends + [few[-1]] * 10007, dtype=I32).cuda()
    few = torch.tensor(few, dtype=I32).cuda()
    loss, counts = fq.moe_balance(l, ids, sequences=ends)
    loss3, counts3 = fq.moe_balance(l, ids, sequences=few)
    assert torch.equal(counts[at], counts3) and int(counts.sum()) == int(counts3.sum())
    # sums of at most T and E positive terms in two orders
    assert bool(((loss[at] - loss3).abs() <= 2 * (T + E) * rl.U * loss3).all())
    rest = torch.ones(len(ends), dtype=torch.bool)
    rest[at] = False
    assert not loss[rest.cuda()].any()
    dloss = torch.linspace(0.5, 1.5, len(ends)).cuda()
    d = fq.moe_route_backward(l, ids, dw, dloss=dloss, counts=counts, sequences=ends)
    assert torch.equal(d, fq.moe_route_backward(l, ids, dw, dloss=dloss[at].contiguous(), counts=counts3, sequences=few))
