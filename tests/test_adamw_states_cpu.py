"""States, masters and parameters of AdamWStates that were given other memory, without a GPU."""
from __future__ import annotations

import pytest
import torch

import fp8_quantization_grouped_amd as fq
from tests.test_adamw_cpu import states
from tests.test_binding_cpu import BF16, calls, gpu, zeros  # noqa: F401

KINDS = ["params", "masters", "exp_avg", "exp_avg_sq", "exp_avg_scales", "exp_avg_sq_scales"]


def made(bits):
    p, m = [zeros(300, dtype=BF16), zeros(0), zeros(4, 4)], [zeros(300), None, None]
    if bits == 8:
        return states(p, m)
    like = lambda: [zeros(*t.shape) for t in p]
    return fq.AdamWStates(p, 32, m, like(), like())


@pytest.mark.parametrize("bits,kind", [(b, k) for b in (8, 32) for k in KINDS if b == 8 or "scales" not in k])
@pytest.mark.parametrize("how", ["data", "entry", "list"])
def test_step_refuses_whatever_was_given_other_memory(calls, bits, kind, how):  # noqa: F811
    """Loaded into the tensor's data, put into the list, or with a list of its own: the step would go on with the
    memory that it knows, and what was loaded would be ignored."""
    s = made(bits)
    grads = [zeros(300), zeros(0), zeros(4, 4)]
    fq.adamw_step(s, grads, 1, 1e-3)
    held = getattr(s, kind)
    loaded = torch.zeros_like(held[0])
    if how == "data":
        held[0].data = loaded
    elif how == "entry":
        held[0] = loaded
    else:
        setattr(s, kind, [loaded] + held[1:])
    with pytest.raises(ValueError, match="other memory"):
        fq.adamw_step(s, grads, 2, 1e-3)
    fq.adamw_step(s, [None] + grads[1:], 2, 1e-3)  # (a tensor that is not stepped is not looked at)
    assert len(calls) == 2


@pytest.mark.parametrize("kind", KINDS)
def test_step_refuses_lists_of_another_length(calls, kind):  # noqa: F811
    for other in (lambda t: t[:-1], lambda t: t + t[-1:]):
        s = made(8)
        setattr(s, kind, other(getattr(s, kind)))
        with pytest.raises(ValueError):
            fq.adamw_step(s, [None, None, zeros(4, 4)], 1, 1e-3)
    assert calls == []


def test_a_master_that_was_added_or_taken_away(calls):  # noqa: F811
    for at, to in ((0, None), (2, zeros(4, 4))):
        s = made(8)
        s.masters[at] = to
        with pytest.raises(ValueError, match="other memory"):
            fq.adamw_step(s, [zeros(300), zeros(0), zeros(4, 4)], 1, 1e-3)
    assert calls == []


def test_states_changed_in_place_are_stepped(calls):  # noqa: F811
    s = made(8)
    for t in s.exp_avg + s.exp_avg_sq_scales:
        t.copy_(torch.ones_like(t))
    s.exp_avg = list(s.exp_avg)
    fq.adamw_step(s, [zeros(300), zeros(0), zeros(4, 4)], 1, 1e-3)
    assert len(calls) == 1
