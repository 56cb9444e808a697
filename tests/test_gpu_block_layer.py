"""The example layer: routing, both products, their gradients and decoding together, against the
same layer in float32 with the bf16 weights."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,I,E,top", [(96, 256, 160, 4, 2), (33, 400, 128, 7, 3)])
def test_layer_against_float32(T, H, I, E, top):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from examples import block_moe_layer as ex
    layer = ex.make(E, H, I, top, seed=T)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    dy = torch.randn(T, H, generator=torch.Generator().manual_seed(2)).cuda()
    y = layer.forward(x)
    dx, dw13, dw2 = layer.backward(dy)
    few = layer.decode(x)

    ids, weights = ex.fq.moe_route(x, layer.router, top)
    xr = x.float().requires_grad_()
    w13, w2 = layer.w13.w.float().requires_grad_(), layer.w2.w.float().requires_grad_()
    want = torch.zeros(T, H, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gate, up = (xr[t] @ w13[e].t()).chunk(2, 1)
        out = (torch.nn.functional.silu(gate) * up) @ w2[e].t()
        want = want.index_add(0, t, out * weights[t, j][:, None])
    want.backward(dy)

    def off(a, b):
        return float((a.float() - b).norm() / b.norm())

    # an e4m3 rounding is at most 2^-4 of a value, about 2^-5.3 in the mean square; each product has
    # two such operands, and a result depends on at most three products one after the other:
    # sqrt(6) 2^-5.3 < 2^-3.9; decoding rounds the weights alone
    assert off(y, want.detach()) < 2.0 ** -3.9
    assert off(dx, xr.grad) < 2.0 ** -3.9
    assert off(dw13, w13.grad) < 2.0 ** -3.9
    assert off(dw2, w2.grad) < 2.0 ** -3.9
    assert off(few, want.detach()) < 2.0 ** -4.4
