"""A mixture-of-experts feed-forward layer on block-scaled FP8 weights: one training step and
decoding, on the same quantized bytes.

    python examples/block_moe_layer.py [--tokens 4096 --hidden 2048 --inner 1408 --experts 64 --top 6]

Training quantizes the expert weights once per step in both layouts, routes the tokens, and runs the
experts' two products and their gradients as grouped products; the activation's and the routing's
gradients are torch operations on their results.  Decoding routes a few tokens and runs the whole
layer on the forward's weight bytes.
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
        ids, weights = fq.moe_route(x, self.router, self.top)
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

    def backward_routing(self, dy):
        """dy float32 [T, H] -> gradients of x [T, H] (through the routing weights) and the router
        [E, H], both float32.  The renormalized weights are a softmax of the chosen logits alone."""
        x, ids, weights, order, o = self.routed
        dw = torch.empty(order.shape, device=dy.device)
        dw[order] = (dy[order // self.top] * o.float()).sum(1)
        dw = dw.view(ids.shape)
        chosen = weights * (dw - (weights * dw).sum(1, keepdim=True))
        dlogits = torch.zeros(x.shape[0], self.router.shape[0], device=dy.device).scatter_(1, ids.long(), chosen)
        return dlogits @ self.router.float(), dlogits.t() @ x.float()

    def decode(self, x):
        """x bf16 [T <= 128, H] -> y bf16 [T, H]."""
        ids, weights = fq.moe_route(x, self.router, self.top)
        return fq.fp8_moe_few_tokens(x, ids, weights, self.w13.forward_bytes, self.w13.scales,
                                     self.w2.forward_bytes, self.w2.scales)


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
    print(f"decoding against the grouped products: {float((y - d).norm() / y.norm()):.3f} "
          "(the products quantize the activations too)")


if __name__ == "__main__":
    main()
