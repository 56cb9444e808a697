"""The AdamW step in 64 bits, with bounds for 32-bit arithmetic, and the random bits that 8-bit states are
rounded by.  Test infrastructure only."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
TINY = 2.0 ** -120


def mix(z):
    """Two rounds of xor-shift and odd product in 32 bits; z int64."""
    z = ((z ^ (z >> 16)) * 0x7F4A7C15) & 0xFFFFFFFF
    z = ((z ^ (z >> 15)) * 0x2C9277B5) & 0xFFFFFFFF
    return z ^ (z >> 16)


def words(seed, index, n):
    key = int(mix(torch.tensor([(seed * 0x9E3779B1 + index) & 0xFFFFFFFF]))[0])
    return mix((torch.arange(n) + key) & 0xFFFFFFFF)


def grid(y, u):
    """The e4m3fn grid's value at or below |y|, or the next one where the rest and u reach a step."""
    y = y.clamp(-448, 448)
    step = torch.exp2((torch.frexp(y)[1].double() - 1).clamp(min=-6) - 3)
    return torch.sign(y) * torch.floor(y.abs() / step + u) * step


def f32(x):
    return float(np.float32(x))


def decode(q, d):
    v = q.cpu().flatten().view(torch.float8_e4m3fn).double()
    return v * d.cpu().double().repeat_interleave(128)[:len(v)]


def step64(p, g, m, v, t, lr, betas, eps, decay, scale=1.0):
    """(p', m', v') and how far 32-bit arithmetic may be from each: every operation and constant U, a root
    and a quotient 2 U."""
    lr, eps, decay = f32(lr), f32(eps), f32(decay)
    g = g * scale
    m1, b = betas[0] * m + (1 - betas[0]) * g, betas[0] * m.abs() + (1 - betas[0]) * g.abs()
    v1 = betas[1] * v + (1 - betas[1]) * g * g
    off_m, off_v = 4 * U * b + TINY, 6 * U * v1 + TINY
    mh, den = m1 / (1 - betas[0] ** t), torch.sqrt(v1 / (1 - betas[1] ** t)) + eps
    d = mh / den
    # corrections 8 U (from a step on the device: its logarithm, exponential and quotient), half of v's error
    off_d = (off_m / (1 - betas[0] ** t)) / den + 24 * U * d.abs()
    p1 = p - lr * (d + decay * p)
    return p1, lr * (off_d + 4 * U * (d.abs() + decay * p.abs())) + 2 * U * (p.abs() + p1.abs()), m1, off_m, v1, off_v


def check_kept(q, d, x, off, word, root):
    """Bytes q and factors d of x in 64 bits, which the call knew up to off."""
    n = len(x)
    pad = lambda a: torch.nn.functional.pad(a, (0, -n % 128)).view(-1, 128)
    amax, slack = pad(x).abs().amax(1), pad(off).amax(1)
    d = d.cpu().double()
    floor = f32(1e-12)
    want = amax.clamp(min=floor) / 448
    assert bool(((d - want).abs() <= slack / 448 + 4 * U * want).all())
    s = (1 / d).repeat_interleave(128)[:n]
    if root:
        word = ((word << 16) | (word >> 16)) & 0xFFFFFFFF
    u = (word >> 12).double() / 2 ** 20
    got = q.cpu().flatten().view(torch.float8_e4m3fn).double()
    ends = []
    for sign in (-1, 1):  # the grid's value only grows with y
        y = x + sign * (off + 6 * U * x.abs())
        e = grid(y * s, u)
        ends.append(torch.where((y > 0) & (e == 0), 2.0 ** -9, e) if root else e)
    assert bool(((got >= ends[0]) & (got <= ends[1])).all())
    if root:
        assert bool((got[x > 2 * off] > 0).all())
