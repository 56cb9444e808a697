"""A mixture-of-experts feed-forward layer on block-scaled FP8 weights, by itself and in its place in a
model: one training step with its update, a prompt and decoding, on the same quantized bytes.

    python examples/block_moe_layer.py [--tokens 4096 --hidden 2048 --inner 1408 --experts 64 --top 6]

Training quantizes the expert weights once per step in both layouts, routes the tokens, and runs the
experts' two products and their gradients as grouped products; the activation's gradient is torch
operations on their results.  Decoding routes a few tokens and runs the whole layer on the forward's
weight bytes.  The block puts the norm with the residual's addition before the layer, the router's
balance loss beside it, and the AdamW step of all of its weights behind its backward pass.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_quantization_grouped_amd as fq  # noqa: E402

FWD, WGRAD = fq.GEMM_FWD_MGROUPED, fq.GEMM_WGRAD_KGROUPED


class Experts:
    """Weights [E, rows, cols] in bf16 and their block-scaled FP8 bytes."""

    def __init__(self, w: torch.Tensor):
        self.w = w
        E, rows, cols = w.shape
        q, q_t, self.scales = fq.fp8_block_quant_weights(w.view(E * rows, cols), E)
        self.forward_bytes = q.unflatten(0, (E, rows))                       # [E, rows, cols]
        self.transposed_bytes = q_t.unflatten(1, (E, rows)).transpose(0, 1)  # [E, cols, rows]

    def product(self, x, offsets):
        """y = x w_e^T, rows grouped by expert; x is (bytes, scales)."""
        return fq.fp8_block_grouped_gemm(FWD, *x, self.forward_bytes, self.scales, offsets)

    def data_gradient(self, dy, offsets):
        """dx = dy w_e."""
        return fq.fp8_block_grouped_gemm(FWD, *dy, self.transposed_bytes,
                                         self.scales.transpose(1, 2), offsets)


def weight_gradient(dy_t, x_t, offsets):
    """dw[e] = dy_e^T x_e [rows, cols] from both sides' transposed bytes."""
    return fq.fp8_block_grouped_gemm(WGRAD, *dy_t, *x_t, offsets)


class Layer:
    def __init__(self, router, w13, w2, top: int):
        """router [E, H]; w13 [E, 2I, H], gate rows first; w2 [E, H, I]; all bf16."""
        self.router, self.top = router, top
        self.w13, self.w2 = Experts(w13), Experts(w2)

    def forward(self, x):
        """x bf16 [T, H] -> y float32 [T, H]; keeps what backward needs."""
        E = self.router.shape[0]
        self.logits = torch.empty(x.shape[0], E, device=x.device)
        ids, weights = fq.moe_route(x, self.router, self.top, logits=self.logits)
        order = torch.argsort(ids.flatten(), stable=True)      # choices grouped by expert
        token = order // self.top
        offsets = torch.cumsum(torch.bincount(ids.flatten(), minlength=E), 0).to(torch.int32)
        share = weights.flatten()[order][:, None]
        rows, rows_t = fq.fp8_block_quant_dual(x[token])
        gu = self.w13.product(rows, offsets).float()
        gate, up = gu.chunk(2, 1)
        h, h_t = fq.fp8_block_quant_dual((torch.nn.functional.silu(gate) * up).to(torch.bfloat16))
        o = self.w2.product(h, offsets)
        self.saved = token, offsets, share, rows_t, gate, up, h_t
        self.routed = x, ids, weights, order, o
        return torch.zeros(x.shape, device=x.device).index_add_(0, token, o.float() * share)

    def backward(self, dy):
        """dy float32 [T, H] -> gradients of x [T, H] (through the experts), w13 and w2."""
        token, offsets, share, x_t, gate, up, h_t = self.saved
        do, do_t = fq.fp8_block_quant_dual((dy[token] * share).to(torch.bfloat16))
        dh = self.w2.data_gradient(do, offsets).float()
        dw2 = weight_gradient(do_t, h_t, offsets)
        s = torch.sigmoid(gate)
        dgu = torch.cat([dh * up * s * (1 + gate * (1 - s)), dh * gate * s], 1).to(torch.bfloat16)
        dgu, dgu_t = fq.fp8_block_quant_dual(dgu)
        dx = self.w13.data_gradient(dgu, offsets).float()
        dw13 = weight_gradient(dgu_t, x_t, offsets)
        return torch.zeros(dy.shape, device=dy.device).index_add_(0, token, dx), dw13, dw2

    def backward_routing(self, dy, **balance):
        """dy float32 [T, H] -> gradients of x [T, H] (through the routing weights) and the router
        [E, H], both float32; balance: dloss, counts and sequences of a balance loss that joins them."""
        x, ids, _, order, o = self.routed
        dw = torch.empty(order.shape, device=dy.device)
        dw[order] = (dy[order // self.top] * o.float()).sum(1)
        dlogits = fq.moe_route_backward(self.logits, ids, dw.view(ids.shape), **balance)
        return dlogits @ self.router.float(), dlogits.t() @ x.float()

    def prompt(self, q, scales, x):
        """x bf16 [T, H] and its rows in 8 bits -> y float32 [T, H]; keeps nothing."""
        ids, weights = fq.moe_route(x, self.router, self.top)
        order = torch.argsort(ids.flatten(), stable=True)
        token = order // self.top
        offsets = torch.cumsum(torch.bincount(ids.flatten(), minlength=self.router.shape[0]), 0).to(torch.int32)
        gate, up = self.w13.product((q[token], scales[:, token]), offsets).float().chunk(2, 1)
        h = fq.fp8_block_quant_rowwise((torch.nn.functional.silu(gate) * up).to(torch.bfloat16))
        o = self.w2.product(h, offsets).float() * weights.flatten()[order][:, None]
        return torch.zeros(x.shape, device=x.device).index_add_(0, token, o)

    def decode(self, x):
        """x bf16 [T <= 128, H] -> y bf16 [T, H]."""
        ids, weights = fq.moe_route(x, self.router, self.top)
        return fq.fp8_moe_few_tokens(x, ids, weights, self.w13.forward_bytes, self.w13.scales,
                                     self.w2.forward_bytes, self.w2.scales)


class Block:
    """The layer behind the norm of a residual stream, and its weights' training."""

    def __init__(self, gain, layer: Layer, bits: int = 8):
        """gain float32 [H], the norm's weight."""
        self.gain, self.layer = gain, layer
        self.states = fq.AdamWStates([gain, layer.router, layer.w13.w, layer.w2.w], bits)
        self.steps = 0

    def forward(self, x, residual, sequences=None):
        """x, residual bf16 [T, H] -> the layer's y float32 [T, H], the stream h = x + residual and the
        balance loss of each sequence."""
        self.normed = fq.fp8_rms_norm(x, self.gain, residual=residual, scaling=None)
        y = self.layer.forward(self.normed.y)
        loss, counts = fq.moe_balance(self.layer.logits, self.layer.routed[1], sequences=sequences)
        self.balance = {"counts": counts, "sequences": sequences}
        return y, self.normed.h, loss

    def backward(self, dy, dh, dloss):
        """Gradients of the three -> that of x and of the residual alike, and those of the weights in the
        states' order."""
        dx, dw13, dw2 = self.layer.backward(dy)
        routing, drouter = self.layer.backward_routing(dy, dloss=dloss, **self.balance)
        dx, dgain = fq.fp8_rms_norm_backward(dx.add_(routing), self.normed.h, self.normed.rstd, self.gain, dh=dh)
        return dx, [dgain, drouter, dw13, dw2]

    def update(self, grads, lr: float):
        """The AdamW step, and the new weights' bytes."""
        self.steps += 1
        fq.adamw_step(self.states, grads, self.steps, lr, betas=(0.9, 0.95), weight_decay=0.1)
        self.layer.w13, self.layer.w2 = Experts(self.layer.w13.w), Experts(self.layer.w2.w)

    def prompt(self, x, residual):
        """A forward that no backward follows: the products read the norm's 8-bit rows."""
        n = fq.fp8_rms_norm(x, self.gain, residual=residual, bf16=True)
        return self.layer.prompt(n.q, n.scales, n.y), n.h

    def decode(self, x, residual):
        """x, residual bf16 [T <= 128, H]."""
        n = fq.fp8_rms_norm(x, self.gain, residual=residual, scaling=None)
        return self.layer.decode(n.y), n.h


def make(experts: int, hidden: int, inner: int, top: int, seed: int = 0) -> Layer:
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    return Layer(normal(experts, hidden, scale=hidden ** -0.5),
                 normal(experts, 2 * inner, hidden, scale=hidden ** -0.5),
                 normal(experts, hidden, inner, scale=inner ** -0.5), top)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inner", 1408), ("experts", 64), ("top", 6)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    layer = make(a.experts, a.hidden, a.inner, a.top)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    few = x[:8].contiguous()

    def timed(f, n=10):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / n * 1e6

    def step():
        y = layer.forward(x)
        dy = torch.ones_like(y)
        return layer.backward(dy), layer.backward_routing(dy)

    print(f"training step, {a.tokens} tokens: {timed(step):.0f} us")
    print(f"decoding 8 tokens: {timed(lambda: layer.decode(few)):.0f} us")
    y, d = layer.forward(few), layer.decode(few).float()
    block = Block(torch.ones(a.hidden, device="cuda"), layer)
    zero, ones = torch.zeros_like(x), torch.full((1,), 1e-2, device="cuda")

    def block_step():
        y, h, _ = block.forward(x, zero)
        block.update(block.backward(torch.full_like(y, 1e-3), None, ones)[1], 1e-5)

    print(f"block: training step with update {timed(block_step):.0f} us, prompt {timed(lambda: block.prompt(x, zero)):.0f} us, "
          f"decoding 8 tokens {timed(lambda: block.decode(few, zero[:8])):.0f} us")
    print(f"decoding against the grouped products: {float((y - d).norm() / y.norm()):.3f} "
          "(the products quantize the activations too)")


if __name__ == "__main__":
    main()
