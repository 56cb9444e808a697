"""Refusals of fp8_rms_norm and fp8_rms_norm_backward, without a GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

import fp8_quantization_grouped_amd as fq
from tests.test_binding_cpu import BF16, F32, U8, calls, gpu, one_row, zeros  # noqa: F401

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p(4096)  # never read: every call here is refused, or has nothing to do


def norm(**kw):
    a = dict(x=P, rows=4, cols=8, ld_x=8, residual=None, ld_res=0, weight=P, wtype=0, eps=1e-6, h=None, ld_h=0, y=None, ld_y=0,
             scaling=2, fmt=1, q=P, ld_q=8, scales=P, ld_s=4, rstd=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return fq.lib().fp8_rms_norm(*a.values())


def back(**kw):
    a = dict(dy=P, ld_dy=8, dh=None, ld_dh=0, grad=0, h=P, rows=4, cols=8, ld_h=8, rstd=P, weight=P, wtype=0, dx=P, ld_dx=8, dw=P,
             ws=P, size=1 << 20, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return fq.lib().fp8_rms_norm_backward(*a.values())


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(ld_x=7), dict(x=None), dict(weight=None), dict(wtype=2), dict(eps=0.0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(scaling=3), dict(fmt=2), dict(fmt=0), dict(q=None), dict(scales=None), dict(ld_q=7), dict(ld_s=3),
    dict(residual=P, ld_res=8), dict(h=P, ld_h=8), dict(residual=P, ld_res=7, h=P, ld_h=8), dict(residual=P, ld_res=8, h=P, ld_h=7),
    dict(residual=P, ld_res=8, h=P, ld_h=9), dict(y=P, ld_y=7), dict(scaling=0), dict(scaling=0, q=None, scales=None),
    dict(scaling=0, q=None, y=P, ld_y=8)])
def test_norm_refuses(kw):
    assert norm(**kw) == INVALID


def test_norm_limits_and_nothing_to_do():
    assert norm(rows=1 << 31, ld_s=1 << 31) == UNSUPPORTED
    assert norm(rows=0, x=None, q=None) == OK and norm(cols=0, x=None) == OK


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(ld_dy=7), dict(dh=P, ld_dh=7), dict(ld_h=7), dict(ld_dx=7), dict(grad=2), dict(wtype=-1),
    dict(dy=None), dict(h=None), dict(rstd=None), dict(weight=None), dict(dx=None), dict(dw=None), dict(ld_dx=9), dict(ws=ctypes.c_void_p(4100)),
    dict(dh=ctypes.c_void_p(8192), ld_dh=8, dx=ctypes.c_void_p(8192), ld_dx=16)])
def test_backward_refuses(kw):
    assert back(**kw) == INVALID


def test_backward_limits():
    assert back(rows=1 << 31) == UNSUPPORTED and back(cols=1 << 31, ld_dy=1 << 31, ld_h=1 << 31, ld_dx=1 << 31) == UNSUPPORTED
    need = fq.fp8_rms_norm_backward_workspace_size(4, 8)
    assert need > 0 and back(size=need - 1) == WORKSPACE and back(ws=None) == WORKSPACE
    assert back(cols=0, dw=None) == OK


def test_binding_refuses(calls):  # noqa: F811
    x, w = zeros(4, 256, dtype=BF16), zeros(256)
    bad = [dict(x=zeros(4, 256)), dict(x=zeros(4, 4, 256, dtype=BF16)), dict(x=torch.zeros(4, 256, dtype=BF16)), dict(weight=zeros(255)),
           dict(weight=zeros(256, dtype=torch.float16)), dict(weight=zeros(512)[::2]), dict(eps=0.0), dict(scaling="tensor"),
           dict(fmt=fq.E4M3FNUZ), dict(scaling="row", fmt=7), dict(residual=zeros(4, 128, dtype=BF16)), dict(h=x),
           dict(scaling=None, q=zeros(4, 256, dtype=U8)), dict(q=zeros(4, 255, dtype=U8)), dict(scales=zeros(4, 2)),
           dict(scaling="row", scales=zeros(4, 1)), dict(rstd=zeros(4, dtype=BF16)), dict(y=zeros(4, 256)),
           dict(q=zeros(4, 256, dtype=U8).view(torch.float8_e4m3fnuz)), dict(residual=x, h=zeros(3, 256, dtype=BF16))]
    for kw in bad:
        with pytest.raises(ValueError):
            fq.fp8_rms_norm(**{"x": x, "weight": w, **kw})
    dy = zeros(4, 256)
    for kw in (dict(dy=x, dh=dy), dict(h=dy), dict(rstd=zeros(3)), dict(dx=x), dict(dweight=zeros(256, dtype=BF16)), dict(weight=zeros(1)),
               dict(workspace=torch.zeros(8)), dict(dy=zeros(4, 256, dtype=torch.float16))):
        with pytest.raises(ValueError):
            fq.fp8_rms_norm_backward(**{"dy": dy, "h": x, "rstd": zeros(4), "weight": w, **kw})
    assert calls == []


def test_a_norm_that_torch_would_record_is_refused(calls):  # noqa: F811
    for which in range(3):
        t = [zeros(4, 256, dtype=BF16), zeros(256), zeros(4, 256, dtype=BF16)]
        t[which].requires_grad_()
        with pytest.raises(ValueError, match="fp8_rms_norm_backward"):
            fq.fp8_rms_norm(t[0], t[1], residual=t[2])
        with torch.no_grad():
            fq.fp8_rms_norm(t[0], t[1], residual=t[2])
    assert len(calls) == 3


def test_one_row_of_any_stride(calls):  # noqa: F811
    for stride in (1, 257, 1 << 34):
        x = one_row(256, stride, BF16)
        fq.fp8_rms_norm(x, zeros(256), residual=x, h=x, bf16=True)
        args = calls[-1][1]
        assert args[3] == args[5] == args[10] == 256
        fq.fp8_rms_norm_backward(x, x, zeros(1), zeros(256), dh=x, dx=x)
        args = calls[-1][1]
        assert args[1] == args[3] == args[8] == args[13] == 256


def test_a_backward_that_torch_would_record_is_refused(calls):  # noqa: F811
    x, w = zeros(4, 256, dtype=BF16), zeros(256).requires_grad_()
    for which in range(2):
        t = [zeros(4, 256), zeros(4, 256)]
        t[which].requires_grad_()
        with pytest.raises(ValueError, match="no gradient"):
            fq.fp8_rms_norm_backward(t[0], x, zeros(4), w, dh=t[1])
    fq.fp8_rms_norm_backward(zeros(4, 256), x, zeros(4), w)  # (a weight that is a parameter is no obstacle)
    ids = zeros(6, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="no gradient"):
        fq.moe_route_backward(zeros(6, 8), ids, zeros(6, 2).requires_grad_())
    assert len(calls) == 1
