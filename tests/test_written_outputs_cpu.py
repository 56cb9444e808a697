"""Tensors that the norm's and the router's calls are given to write: torch learns that their values changed, without
a GPU.  A product that has saved such a tensor for its gradient would else take the new values for the old ones."""
from __future__ import annotations

import pytest
import torch

import fp8_quantization_grouped_amd as fq
from tests.test_binding_cpu import BF16, F32, U8, calls, gpu, zeros  # noqa: F401

I32 = torch.int32
T, H, E, K = 4, 256, 8, 2


def norm(**given):
    fq.fp8_rms_norm(*given.pop("x", [zeros(T, H, dtype=BF16)]), zeros(H), **{"residual": zeros(T, H, dtype=BF16), **given})


def back(**given):
    fq.fp8_rms_norm_backward(given.pop("dy", zeros(T, H)), zeros(T, H, dtype=BF16), zeros(T), zeros(H), **given)


def balance(**given):
    fq.moe_balance(zeros(T, E), zeros(T, K, dtype=I32), **given)


def route_back(**given):
    fq.moe_route_backward(given.pop("logits", zeros(T, E)), zeros(T, K, dtype=I32), zeros(T, K), **given)


def route(**given):
    fq.moe_route(zeros(T, H, dtype=BF16), zeros(E, H, dtype=BF16), K, **given)


CASES = [(norm, "h", (T, H), BF16), (norm, "y", (T, H), BF16), (norm, "q", (T, H), U8), (norm, "scales", (2, T), F32), (norm, "rstd", (T,), F32),
         (back, "dx", (T, H), F32), (back, "dweight", (H,), F32), (balance, "loss", (1,), F32), (balance, "counts", (1, E), I32),
         (route_back, "dlogits", (T, E), F32), (route, "logits", (T, E), F32)]


@pytest.mark.parametrize("call,name,shape,dtype", CASES)
def test_a_given_output_is_changed(calls, call, name, shape, dtype):  # noqa: F811
    t = zeros(*shape, dtype=dtype)
    before = t._version
    call(**{name: t})
    assert t._version == before + 1 and len(calls) == 1
    with torch.inference_mode():  # such a tensor has no version, and nothing saves it
        t = zeros(*shape, dtype=dtype)
        call(**{name: t})
    assert len(calls) == 2


@pytest.mark.parametrize("replace", ["x", "residual", "dy", "dh", "logits"])
def test_a_replaced_operand_that_torch_has_saved(calls, replace):  # noqa: F811
    dtype = BF16 if replace in ("x", "residual") else F32
    t = zeros(T, E if replace == "logits" else H, dtype=dtype)
    w = torch.ones(t.shape, dtype=dtype, requires_grad=True)
    loss = (w * t).sum()
    {"x": lambda: norm(x=[t], h=t), "residual": lambda: norm(residual=t, h=t), "dy": lambda: back(dy=t, dx=t), "dh": lambda: back(dh=t, dx=t),
     "logits": lambda: route_back(logits=t, dlogits=t)}[replace]()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_what_is_only_read_is_not_changed(calls):  # noqa: F811
    x, r, g = zeros(T, H, dtype=BF16), zeros(T, H, dtype=BF16), zeros(H)
    fq.fp8_rms_norm(x, g, residual=r)
    fq.fp8_rms_norm(x, g)
    dy, dh, s = zeros(T, H), zeros(T, H), zeros(T)
    fq.fp8_rms_norm_backward(dy, x, s, g, dh=dh)
    l, ids, dw, dl, c = zeros(T, E), zeros(T, K, dtype=I32), zeros(T, K), zeros(1), zeros(1, E, dtype=I32)
    fq.moe_balance(l, ids)
    fq.moe_route_backward(l, ids, dw, dloss=dl, counts=c)
    assert [t._version for t in (x, r, g, dy, dh, s, l, ids, dw, dl, c)] == [0] * 11 and len(calls) == 5


def test_a_refused_call_changes_nothing(calls):  # noqa: F811
    x = zeros(T, H, dtype=BF16)
    with pytest.raises(ValueError):
        norm(h=x, y=zeros(T, H))
    assert x._version == 0 and calls == []
