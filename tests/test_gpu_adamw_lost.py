"""Gradients that 32 bits cannot hold the squares of, infinite ones and NaN, beside ordinary ones: what happens to an
element stays with it."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_adamw import BF16, F32, fq, normal, states_of  # noqa: F401

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def run(fq, bits, n, at, values, grad, param, shift=0):
    """Three steps of three tensors: the first with values in the middle one's gradient at the places at; None for the
    run that they are held against, where nothing is there: no gradient and no state."""
    masters = [normal(k, i, shift=shift) for i, k in enumerate((300, n, 129))] if param == "master" else None
    params = [m.to(BF16) for m in masters] if masters else [normal(k, i, BF16 if param == "bf16" else F32, shift=shift) for i, k in enumerate((300, n, 129))]
    s = states_of(fq, params, bits, masters)
    if values is None:
        s.exp_avg[1].view(-1)[at] = 0
        s.exp_avg_sq[1].view(-1)[at] = 0
    after = []
    for t in (5, 6, 7):
        grads = [normal(k, 100 * t + i, grad, 2e-3, shift) for i, k in enumerate((300, n, 129))]
        if values is None:
            grads[1][at] = 0
        elif t == 5:
            grads[1][at] = torch.tensor(values, device="cuda").to(grad)
        fq.adamw_step(s, grads, t, 1e-2, betas=(0.9, 0.999), seed=3)
        lists = [s.params, s.exp_avg, s.exp_avg_sq] + ([s.exp_avg_scales, s.exp_avg_sq_scales] if bits == 8 else []) + ([s.masters] if masters else [])
        after.append([[x.clone() for x in tensors] for tensors in lists])
    return after


PLACES = [([5], [INF]), ([131], [NAN]), ([260], [1e25]), ([0, 127, 128, 640], [-INF, NAN, INF, -1e30]), ([700, 701, 702, 703], [1e25, -1e25, NAN, INF]),
          (list(range(384, 512)), [INF, NAN, -INF, 3e30] * 32), ([2176, 2177, 4223, 4225], [INF, NAN, 1e28, -INF]), ([4999], [INF]), ([4992], [NAN])]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("grad,param", [(F32, "fp32"), (BF16, "bf16"), (F32, "master")])
@pytest.mark.parametrize("shift", [0, 1])
def test_what_32_bits_cannot_hold_stays_with_its_element(fq, bits, grad, param, shift):  # noqa: F811
    n = 5000
    for at, values in PLACES:
        if shift and len(at) > 4:
            continue
        bare, mine = run(fq, bits, n, at, None, grad, param, shift), run(fq, bits, n, at, values, grad, param, shift)
        rest = torch.ones(n, dtype=torch.bool, device="cuda")
        rest[at] = False
        for step, (a, b) in enumerate(zip(bare, mine)):
            for kind, (x, y) in enumerate(zip(a, b)):
                assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2])
                same = slice(None) if x[1].numel() != n else rest  # factors: all of them
                if bits == 8 or x[1].numel() == n:
                    assert torch.equal(x[1][same], y[1][same]), (at, step, kind)
                    assert bool(torch.isfinite(y[1][same].float()).all())
            p, m, v = b[0][1][at].float(), b[1][1][at], b[2][1][at]
            finite = torch.isfinite(torch.tensor(values, device="cuda"))
            assert bool(torch.isnan(p[~finite]).all())
            if bits == 8:  # none of these looks like a state again
                assert bool(((m & 127) == 127).all()) and bool(((v & 127) == 127).all())
                assert step == 0 or bool(torch.isnan(p).all())
            else:
                assert not bool(torch.isfinite(v).any())


def test_largest_gradients_whose_squares_are_held(fq):  # noqa: F811
    """Just inside the range nothing is lost: states and factors are finite, and the step is the formula's."""
    from tests.test_gpu_adamw import check, values
    for big in (1e18, -5e20, 1e19):
        params = [normal(400, 1)]
        s = states_of(fq, params, 8)
        grads = [normal(400, 2, scale=2e-3)]
        grads[0][200] = big
        before = values(s)
        fq.adamw_step(s, grads, 5, 1e-2)
        check(s, before, grads, 5, 1e-2, (0.9, 0.999), 1e-8, 0.01)
        assert bool(torch.isfinite(s.exp_avg_scales[0]).all()) and bool(torch.isfinite(s.exp_avg_sq_scales[0]).all())


def test_a_captured_step_with_lost_elements(fq):  # noqa: F811
    """Replays, of which the second has an infinite gradient, against the same steps made eagerly."""
    def fresh():
        p = [normal(3000, 1, BF16), normal(700, 2)]
        return states_of(fq, p, 8), [normal(3000, 3, BF16, 1e-2), normal(700, 4, scale=1e-2)]

    (a, ga), (b, gb) = fresh(), fresh()
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fq.adamw_step(a, ga, step, 1e-2)
    for t in range(1, 5):
        step.fill_(t)
        for x, y in zip(ga, gb):
            x.normal_(generator=torch.Generator("cuda").manual_seed(t))
            if t == 2:
                x[100] = INF
            y.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        fq.adamw_step(b, gb, step, 1e-2)
        for x, y in zip(a.exp_avg + a.exp_avg_sq + a.exp_avg_scales + a.exp_avg_sq_scales, b.exp_avg + b.exp_avg_sq + b.exp_avg_scales + b.exp_avg_sq_scales):
            assert torch.equal(x, y), t
        for x, y in zip(a.params, b.params):
            assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x.nan_to_num(), y.nan_to_num())
