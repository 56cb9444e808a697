"""Block-scaled FP8 (blocks of 128) in 64 bits on the CPU, from the definition: what the block
quantizers, the block-scaled products and the mixture-of-experts layer are tested against.

The format holds two intermediate values in 32 bits, the multiplier 448 / max and the product of
an element with it; everything else here is float64.  Test infrastructure only.
"""
from __future__ import annotations

import numpy as np
import torch

B = 128


def held32(v):
    return v.float().double()


def grid(v):
    """Nearest e4m3fn value, ties to even, saturating; -0.0 keeps its sign."""
    v = v.clamp(-448.0, 448.0)
    e = torch.frexp(v.abs())[1].double() - 1
    step = torch.exp2(e.clamp(min=-6.0) - 3)
    return torch.copysign(torch.round(v.abs() / step) * step, v)


def to_bytes(values):
    """e4m3fn bytes of values on the grid."""
    return values.to(torch.float8_e4m3fn).view(torch.uint8)


def decode(q):
    return q.cpu().view(torch.float8_e4m3fn).double()


def _spread(d, dim, n):
    return d.repeat_interleave(B, dim).narrow(dim, 0, n)


def _max(x, dim):
    pad = -x.shape[dim] % B
    x = torch.nn.functional.pad(x.abs(), (0, pad) if dim == 1 else (0, 0, 0, pad))
    return x.unflatten(dim, (-1, B)).amax(dim + 1)


def quant(x, dim):
    """(bytes like x, factors d) of x [R, C] in blocks along dim."""
    x = x.cpu().double()
    s = held32(448.0 / _max(x, dim).clamp(min=float(np.float32(1e-12))))
    q = grid(held32(x * _spread(s, dim, x.shape[dim])))
    return to_bytes(q), held32(1.0 / s)


def quant_rowwise(x):
    q, d = quant(x, 1)
    return q, d.t().contiguous()


def quant_colwise(x):
    q, d = quant(x, 0)
    return q.t().contiguous(), d


def quant_square(w):
    x = w.cpu().double()
    s = held32(448.0 / _max(_max(x, 1), 0).clamp(min=float(np.float32(1e-12))))
    q = grid(held32(x * _spread(_spread(s, 0, x.shape[0]), 1, x.shape[1])))
    return to_bytes(q), held32(1.0 / s)


def real_rows(q, d):
    """What bytes q [rows, cols] with factors d [column blocks, rows] stand for."""
    return decode(q) * _spread(d.cpu().double().t(), 1, q.shape[1])


def real_square(q, d):
    """What bytes q [R, C] with factors d [row blocks, column blocks] stand for."""
    return decode(q) * _spread(_spread(d.cpu().double(), 0, q.shape[0]), 1, q.shape[1])


def product(a, b):
    """a @ b.T and the sum of its terms' magnitudes."""
    return a @ b.t(), a.abs() @ b.abs().t()


def product_bound(exact, mags, dtype):
    """How far a block-scaled product may be from the exact one.  The matrix cores add each 8
    products in fixed point whose last bit is 2^-13 of a power of two at most the largest of the 8,
    each cut off toward zero: at most 8 * 2^-13 of that largest, so 2^-10 of the magnitudes' sum.
    The 32-bit accumulation and factors add at most 2^-20 of it (128-element sums, two factors
    and one fused sum per block, contractions up to 2^14), the output type half a step."""
    return 2.0 ** -10 * mags + 2.0 ** -20 * mags + torch.finfo(dtype).eps / 2 * exact.abs() * 1.01
