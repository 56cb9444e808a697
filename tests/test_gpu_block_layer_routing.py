"""The example layer's routing gradient in 64 bits: against autograd and differences of
sum(dY * Y), Y = sum_j w[t,j] o[t,j] with the experts' outputs o that the forward left behind and the
weights as a function of x and the router.  (How far o is from exact is for the layer's own test.)"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,I,E,top", [(96, 256, 160, 4, 2), (33, 400, 128, 7, 3), (5, 128, 128, 3, 1), (1, 256, 128, 4, 4)])
def test_routing_gradient(T, H, I, E, top):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from examples import block_moe_layer as ex
    layer = ex.make(E, H, I, top, seed=T)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    dy = torch.randn(T, H, generator=torch.Generator().manual_seed(2)).cuda()
    layer.forward(x)
    got_x, got_r = layer.backward_routing(dy)
    assert got_x.shape == (T, H) and got_r.shape == (E, H)

    _, ids, _, order, o = layer.routed
    ids, g64 = ids.long(), dy.double()
    rows = torch.empty(T * top, H, dtype=torch.float64, device="cuda")
    rows[order] = o.double()  # row t * top + j: what expert ids[t, j] made of token t
    rows = rows.view(T, top, H)

    def loss(x, router):
        weights = torch.softmax(torch.gather(x @ router.t(), 1, ids), 1)
        return ((weights[:, :, None] * rows).sum(1) * g64).sum()

    xr, rr = x.double().requires_grad_(), layer.router.double().requires_grad_()
    loss(xr, rr).backward()

    # In 32 bits: dw sums H products; a logit sums H products, and its error is twice a weight's, with a few
    # units in the last place for exponential, sum and quotient; the last products sum E and T terms.
    u = 2.0 ** -24
    ax, ar = x.double().abs(), layer.router.double().abs()
    with torch.no_grad():
        w = torch.softmax(torch.gather(xr @ rr.t(), 1, ids), 1)
        mag = (g64.abs()[:, None, :] * rows.abs()).sum(2)
        mag = w * (mag + (w * mag).sum(1, keepdim=True))
        off_w = 2 * (H * u * (ax @ ar.t()).amax(1, keepdim=True)) + 16 * u
        spread = lambda v: torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, ids, v)
        off, mag = spread(mag * ((H + top + 8) * u + 2 * off_w)), spread(mag)
        assert bool(((got_x.double() - xr.grad).abs() <= off @ ar + (E + 2) * u * (mag @ ar) + 1e-30).all())
        assert bool(((got_r.double() - rr.grad).abs() <= off.t() @ ax + (T + 2) * u * (mag.t() @ ax) + 1e-30).all())

        v = torch.randn(E, H, generator=torch.Generator().manual_seed(3), dtype=torch.float64).cuda()
        v /= v.norm()
        diff = (loss(xr, rr + 1e-5 * v) - loss(xr, rr - 1e-5 * v)) / 2e-5
        slope = (got_r.double() * v).sum()
        # a difference over 1e-5 in a logit of slope at most |x| = 30 is off by about (3e-4)^2
        assert abs(float(slope - diff)) <= float((off.t() @ ax * v.abs()).sum()) + 1e-6 * float((mag.t() @ ax * v.abs()).sum())
