"""Measured cases of the block-scaled FP8 operators: quantizers with one scale per block of 128,
the grouped products on their bytes (forward, both gradients) and a mixture-of-experts layer for
a few tokens on the same weight format.

Every block shares s = 448 / max(amax, 1e-12), held in 32 bits; an element is the e4m3fn value
nearest to x * s, that product held in 32 bits too; the block's stored factor d = 1 / s gives x
back.  Activations have
blocks of 1 x 128 along the contraction, weights blocks of 128 x 128.
"""
import math

import numpy as np
import torch

own = False

FMAX, EPS, BLOCK = 448.0, 1e-12, 128


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest MoE layer of the configurations: launch latency
        {"name": "forward, 4 small experts", "kind": "forward", "groups": 4, "M": 1024, "N": 512, "K": 256},
        # ragged everything: contraction ends inside a block, columns inside a tile, few rows a group
        {"name": "forward, odd sizes", "kind": "forward", "groups": 7, "M": 1333, "N": 1111, "K": 2064},
        # the feed-forward product of a dense 8B model, one group
        {"name": "forward, dense feed-forward", "kind": "forward", "groups": 1, "M": 8192, "N": 14336, "K": 4096},
        # routed tokens of 64 fine-grained experts
        {"name": "forward, 64 experts", "kind": "forward", "groups": 64, "M": 49152, "N": 1408, "K": 2048},
        # a training step's backward on odd row counts: both gradients of one expert layer
        {"name": "backward, odd sizes", "kind": "backward", "groups": 7, "M": 1333, "N": 1104, "K": 2064},
        # the backward of one GPU's slice of a large MoE layer
        {"name": "backward, 32 large experts", "kind": "backward", "groups": 32, "M": 16384, "N": 2048, "K": 7168},
        # both layouts of an activation matrix, for the forward and the weight gradient
        {"name": "activations, both layouts", "kind": "activations", "M": 16384, "K": 7168},
        # both layouts of the expert weights, once per optimizer step
        {"name": "weights, both layouts", "kind": "weights", "groups": 64, "N": 1408, "K": 2048},
        # one token decoded: its 8 experts' weights are all that counts
        {"name": "layer, 1 token", "kind": "layer", "T": 1, "H": 7168, "I": 2048, "E": 32, "top": 8, "scoring": "sigmoid"},
        # a small batch over fine-grained experts
        {"name": "layer, 5 tokens, 64 experts", "kind": "layer", "T": 5, "H": 2048, "I": 1408, "E": 64, "top": 6, "scoring": "softmax"},
        # a decode batch in which every expert has work
        {"name": "layer, 64 tokens", "kind": "layer", "T": 64, "H": 7168, "I": 2048, "E": 32, "top": 8, "scoring": "sigmoid"},
        # the smallest layer
        {"name": "layer, 2 tokens, 4 experts", "kind": "layer", "T": 2, "H": 256, "I": 512, "E": 4, "top": 2, "scoring": "softmax"},
    ]


def _spread(rng, lo, hi, step=1):
    return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step)


def draw(rng):
    kind = rng.choice(["forward", "backward", "activations", "weights", "layer", "layer"])
    if kind in ("forward", "backward"):
        while True:
            c = {"kind": kind, "groups": _spread(rng, 1, 64), "M": _spread(rng, 1, 32768),
                 "N": _spread(rng, 64, 8192, 1 if kind == "forward" else 16), "K": _spread(rng, 64, 8192, 16)}
            if c["M"] * c["N"] * c["K"] <= 1.5e11 and c["groups"] * c["N"] * c["K"] <= 4e8:
                return c
    if kind == "activations":
        while True:
            c = {"kind": kind, "M": _spread(rng, 1, 32768), "K": _spread(rng, 64, 8192, 8)}
            if c["M"] * c["K"] <= 1.1e8:
                return c
    if kind == "weights":
        while True:
            c = {"kind": kind, "groups": _spread(rng, 1, 64), "N": _spread(rng, 64, 4096, 8), "K": _spread(rng, 64, 8192, 16)}
            if c["groups"] * c["N"] * c["K"] <= 1.8e8:
                return c
    while True:
        c = {"kind": kind, "T": _spread(rng, 1, 64), "H": _spread(rng, 256, 7168, 16), "I": _spread(rng, 128, 4096, 16),
             "E": _spread(rng, 4, 128), "top": rng.randint(1, 8), "scoring": rng.choice(["softmax", "sigmoid"])}
        if c["top"] <= c["E"] and 3 * c["E"] * c["H"] * c["I"] <= 1.4e9:
            return c


# ------------------------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)


def _activations(gen, rows, cols):
    """Unit normals with one value in a thousand 30 times as large, as a few channels' are."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x = torch.where(torch.rand(rows, cols, generator=gen, device="cuda") < 1e-3, x * 30, x)
    return x.to(torch.bfloat16)


def _group_sizes(seed, groups, rows):
    """Rows of each group: skewed popularity in a shuffled order, empty groups now and then."""
    rs = np.random.RandomState(seed % (1 << 31))
    p = 1.0 / np.arange(1, groups + 1)
    p = p[rs.permutation(groups)]
    return [int(v) for v in rs.multinomial(rows, p / p.sum())]


def _offsets(sizes):
    return torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = _generator(seed)
    kind = case["kind"]
    if kind == "forward":
        G, M, N, K = case["groups"], case["M"], case["N"], case["K"]
        sizes = _group_sizes(seed, G, M)
        wq, ws = _quantize_square(_normal(gen, G, N, K, scale=0.02))
        return {"case": case, "x": _activations(gen, M, K), "w": wq, "w_scales": ws, "sizes": sizes, "offsets": _offsets(sizes)}
    if kind == "backward":
        G, M, N, K = case["groups"], case["M"], case["N"], case["K"]
        sizes = _group_sizes(seed, G, M)
        wq, ws = _quantize_square(_normal(gen, G, N, K, scale=0.02))
        # the bytes that the forward left behind: the weights' transposed layout [K][G * N] and
        # the activations' [K][M], its rows padded to whole 16 bytes
        wt = wq.permute(2, 0, 1).reshape(K, G * N).contiguous()
        xq, xs = _quantize_columns(_activations(gen, M, K))
        return {"case": case, "dy": _normal(gen, M, N, scale=1e-3), "w_t": wt, "w_scales": ws, "x_t": _padded(xq), "x_scales": xs,
                "sizes": sizes, "offsets": _offsets(sizes)}
    if kind == "activations":
        return {"case": case, "x": _activations(gen, case["M"], case["K"])}
    if kind == "weights":
        return {"case": case, "w": _normal(gen, case["groups"] * case["N"], case["K"], scale=0.02)}
    T, H, I, E = case["T"], case["H"], case["I"], case["E"]
    w13, s13 = _quantize_square(_normal(gen, E, 2 * I, H, scale=0.02))
    w2, s2 = _quantize_square(_normal(gen, E, H, I, scale=0.02))
    state = {"case": case, "x": _normal(gen, T, H), "router": _normal(gen, E, H, scale=H ** -0.5),
             "w13": w13, "s13": s13, "w2": w2, "s2": s2, "bias": None}
    if case["scoring"] == "sigmoid":  # the balancing bias that such routers add for the choice
        state["bias"] = torch.randn(E, generator=gen, device="cuda") * 0.1
    return state


def _padded(q_t):
    """The same [rows, cols] bytes with rows that start on 16 bytes."""
    out = torch.zeros(q_t.shape[0], -(-q_t.shape[1] // 16) * 16, dtype=torch.uint8, device="cuda")
    out[:, :q_t.shape[1]] = q_t
    return out[:, :q_t.shape[1]]


# ------------------------------------------------------------------------------- plain forms

def _blocks(x, dim):
    """x in 32 bits with dimension dim cut into blocks of 128, the last filled up with zeros."""
    x = x.float()
    pad = [0, 0] * (x.dim() - 1 - dim) + [0, -x.shape[dim] % BLOCK]
    return torch.nn.functional.pad(x, pad).unflatten(dim, (-1, BLOCK))


def _scale(amax):
    # a quotient of two tensors: a number over a tensor is the number times a rounded reciprocal
    return torch.full_like(amax, FMAX) / torch.clamp(amax, min=EPS)


def _encode(y):
    return torch.clamp(y, -FMAX, FMAX).to(torch.float8_e4m3fn)


def _quantize_rows(x):
    """Blocks of 128 columns: bytes [rows, cols], factors [column blocks, rows]."""
    b = _blocks(x, 1)
    s = _scale(b.abs().amax(2))
    q = _encode((b * s[:, :, None]).flatten(1)[:, :x.shape[1]])
    return q.contiguous().view(torch.uint8), (1.0 / s).t().contiguous()


def _quantize_columns(x):
    """Blocks of 128 rows, transposed: bytes [cols, rows], factors [row blocks, cols]."""
    b = _blocks(x, 0)
    s = _scale(b.abs().amax(1))
    q = _encode((b * s[:, None, :]).flatten(0, 1)[:x.shape[0]])
    return q.view(torch.uint8).t().contiguous(), 1.0 / s


def _quantize_square(w):
    """Blocks of 128 x 128 of each matrix of w [G, R, C]: bytes like w, factors [G, row blocks, column blocks]."""
    G, R, C = w.shape
    b = _blocks(_blocks(w, 2).flatten(2, 3), 1).unflatten(3, (-1, BLOCK))  # [G, rb, 128, cb, 128]
    s = _scale(b.abs().amax((2, 4)))
    q = _encode(b * s[:, :, None, :, None]).view(torch.uint8)
    return q.flatten(3, 4).flatten(1, 2)[:, :R, :C].contiguous(), 1.0 / s


def _values(q):
    return q.view(torch.float8_e4m3fn).float()


def _dequantize_square(q, d):
    d = d.repeat_interleave(BLOCK, 1)[:, :q.shape[1]].repeat_interleave(BLOCK, 2)[:, :, :q.shape[2]]
    return _values(q) * d


def _dequantize_rows(q, d):
    """q [rows, cols] with factors [column blocks, rows]."""
    return _values(q) * d.t().repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _plain_forward(s):
    x = _dequantize_rows(*_quantize_rows(s["x"]))
    w = _dequantize_square(s["w"], s["w_scales"])
    return torch.cat([a @ b.t() for a, b in zip(x.split(s["sizes"]), w)]).to(torch.bfloat16)


def _plain_backward(s):
    c = s["case"]
    dy = _dequantize_rows(*_quantize_rows(s["dy"]))
    w = _dequantize_square(s["w_t"].unflatten(1, (c["groups"], c["N"])).permute(1, 2, 0).contiguous(), s["w_scales"])
    dx = torch.cat([a @ b for a, b in zip(dy.split(s["sizes"]), w)])
    dy_t = _dequantize_rows(*_quantize_columns(s["dy"]))  # [N, M]: token blocks are its column blocks
    x_t = _dequantize_rows(s["x_t"].contiguous(), s["x_scales"])
    dw = torch.stack([a @ b.t() for a, b in zip(dy_t.split(s["sizes"], 1), x_t.split(s["sizes"], 1))])
    return {"dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}


def _plain_route(x, router, top, bias, scoring):
    logits = x.float() @ router.float().t()
    scores = torch.sigmoid(logits) if scoring == "sigmoid" else torch.exp(logits - logits.amax(1, keepdim=True))
    if scoring == "softmax":
        scores = scores / scores.sum(1, keepdim=True)
    choice = logits if bias is None else scores + bias
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :top]  # ties: the lowest index
    w = torch.gather(scores, 1, ids)
    return ids, w / w.sum(1, keepdim=True)


def _plain_layer(s):
    c = s["case"]
    T, I, E, top = c["T"], c["I"], c["E"], c["top"]
    x = s["x"].float()
    ids, weights = _plain_route(s["x"], s["router"], top, s["bias"], c["scoring"])
    if T * top <= E:  # each chosen expert's weights by themselves
        at = ids.flatten()
        w13 = _dequantize_square(s["w13"][at], s["s13"][at])
        h = torch.matmul(w13, x.repeat_interleave(top, 0)[:, :, None])
        h = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
        o = torch.matmul(_dequantize_square(s["w2"][at], s["s2"][at]), h)
        y = (o.view(T, top, -1) * weights[:, :, None]).sum(1)
    else:  # all experts for all tokens, and the chosen ones' sum
        h = torch.matmul(_dequantize_square(s["w13"], s["s13"]), x.t())
        h = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
        share = torch.zeros(T, E, device=x.device).scatter_(1, ids, weights)
        y = (torch.matmul(_dequantize_square(s["w2"], s["s2"]), h) * share.t()[:, None, :]).sum(0).t()
    return {"y": y.to(torch.bfloat16), "ids": ids.to(torch.int32), "weights": weights}


def _as_values(q, d, q_t, d_t):
    """Bytes as the 8-bit values that they are, beside their factors."""
    return {"q": q.view(torch.float8_e4m3fn), "scales": d, "q_t": q_t.contiguous().view(torch.float8_e4m3fn), "scales_t": d_t}


def _plain_weights(s):
    c = s["case"]
    q, d = _quantize_square(s["w"].view(c["groups"], c["N"], c["K"]))
    q = q.view(-1, c["K"])
    return _as_values(q, d, q.t(), None)


# ---------------------------------------------------------------------------------- one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(state, kind)
    if kind == "forward":
        return _plain_forward(state)
    if kind == "backward":
        return _plain_backward(state)
    if kind == "activations":
        return _as_values(*_quantize_rows(state["x"]), *_quantize_columns(state["x"]))
    if kind == "weights":
        return _plain_weights(state)
    return _plain_layer(state)


def _own(s, kind):
    import fp8_quantization_grouped_amd as fq
    c = s["case"]
    if kind == "forward":
        q, d = fq.fp8_block_quant_rowwise(s["x"])
        return fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q, d, s["w"], s["w_scales"], s["offsets"])
    if kind == "backward":
        (q, d), (q_t, d_t) = fq.fp8_block_quant_dual(s["dy"])
        w_t = s["w_t"].view(c["K"], c["groups"], c["N"]).transpose(0, 1)  # [G, K, N]: the data gradient's operand
        dx = fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, q, d, w_t, s["w_scales"].transpose(1, 2), s["offsets"])
        dw = fq.fp8_block_grouped_gemm(fq.GEMM_WGRAD_KGROUPED, q_t, d_t, s["x_t"], s["x_scales"], s["offsets"])
        return {"dx": dx, "dw": dw}
    if kind == "activations":
        (q, d), (q_t, d_t) = fq.fp8_block_quant_dual(s["x"])
        return {"q": q.view(torch.float8_e4m3fn), "scales": d, "q_t": q_t.view(torch.float8_e4m3fn), "scales_t": d_t}
    if kind == "weights":
        q, q_t, d = fq.fp8_block_quant_weights(s["w"], c["groups"])
        return {"q": q.view(torch.float8_e4m3fn), "scales": d, "q_t": q_t.view(torch.float8_e4m3fn), "scales_t": None}
    ids, weights = fq.moe_route(s["x"], s["router"], c["top"], bias=s["bias"], scoring=c["scoring"])
    y = fq.fp8_moe_few_tokens(s["x"], ids, weights, s["w13"], s["s13"], s["w2"], s["s2"])
    return {"y": y, "ids": ids, "weights": weights}


# -------------------------------------------------------------------------------- their work

def _ceil(a, b):
    return -(-a // b)


def work(case):
    kind = case["kind"]
    if kind in ("forward", "backward"):
        G, M, N, K = case["groups"], case["M"], case["N"], case["K"]
        w = G * N * K + 4 * G * _ceil(N, BLOCK) * _ceil(K, BLOCK)
        if kind == "forward":  # x, the weights, y
            return {"bytes": 2 * M * K + w + 2 * M * N, "flops": 2 * M * N * K}
        # dy, the weights, the activations' bytes, dx, dw
        x_t = M * K + 4 * _ceil(M, BLOCK) * K
        return {"bytes": 2 * M * N + w + x_t + 2 * M * K + 2 * G * N * K, "flops": 4 * M * N * K}
    if kind == "activations":
        M, K = case["M"], case["K"]
        return {"bytes": 4 * M * K + 4 * (M * _ceil(K, BLOCK) + K * _ceil(M, BLOCK)), "flops": 4 * M * K}
    if kind == "weights":
        n = case["groups"] * case["N"] * case["K"]
        return {"bytes": 4 * n + 4 * case["groups"] * _ceil(case["N"], BLOCK) * _ceil(case["K"], BLOCK), "flops": 3 * n}
    T, H, I, E, top = case["T"], case["H"], case["I"], case["E"], case["top"]
    experts = E * (1 - (1 - top / E) ** T)  # expected number that some token chooses
    w = 3 * H * I + 12 * _ceil(H, BLOCK) * _ceil(I, BLOCK)
    return {"bytes": int(experts * w) + 2 * E * H + 4 * T * H + 8 * T * top, "flops": 2 * T * (3 * top * H * I + E * H)}


# --------------------------------------------------------------------------- in 64 bits, apart

def _grid64(v):
    """Nearest e4m3fn value (ties to even) of v in 64 bits, cut off at the largest."""
    v = v.clamp(-448.0, 448.0)
    e = torch.frexp(v.abs())[1].to(torch.float64) - 1
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return torch.round(v / step) * step


def _block_max64(x, dim):
    """Largest magnitude of x [R, C] over blocks of 128 along dim, given for every element."""
    n = x.shape[dim]
    at = torch.arange(n, device=x.device) // 128
    shape = list(x.shape)
    shape[dim] = int(at[-1]) + 1
    index = at[:, None].expand_as(x) if dim == 0 else at[None, :].expand_as(x)
    m = torch.zeros(shape, dtype=torch.float64, device=x.device).scatter_reduce(dim, index, x.abs(), "amax")
    return m.clamp(min=1e-12)


def _held32(v):
    """The 32-bit value nearest to v.  The format says that 448 / max and x times it are held in 32
    bits: bf16 values on a border of the 8-bit grid are frequent, and there these two roundings
    decide."""
    return v.float().double()


def _scale64(m):
    return _held32(448.0 / m)


def _quantized64(x, dim):
    """(values on the 8-bit grid, block factors) of x along dim."""
    x = x.double()
    s = _scale64(_block_max64(x, dim))
    every = s.repeat_interleave(128, dim).narrow(dim, 0, x.shape[dim])
    return _grid64(_held32(x * every)), 1.0 / s


def _real64(x, dim):
    q, d = _quantized64(x, dim)
    return q * d.repeat_interleave(128, dim).narrow(dim, 0, x.shape[dim])


def _square64(q, d):
    """What bytes q [R, C] with factors d [row blocks, column blocks] stand for."""
    r = torch.arange(q.shape[0], device=q.device) // 128
    c = torch.arange(q.shape[1], device=q.device) // 128
    return q.view(torch.float8_e4m3fn).double() * d.double()[r][:, c]


def _exact_grouped(case, s):
    ends = [0] + [int(v) for v in np.cumsum(s["sizes"])]
    G, M, N, K = case["groups"], case["M"], case["N"], case["K"]
    if case["kind"] == "forward":
        x = _real64(s["x"], 1)
        y = torch.empty(M, N, dtype=torch.float64, device="cuda")
        for g in range(G):
            y[ends[g]:ends[g + 1]] = x[ends[g]:ends[g + 1]] @ _square64(s["w"][g], s["w_scales"][g]).t()
        return y
    dy_rows, dy_columns = _real64(s["dy"], 1), _real64(s["dy"], 0)
    t = torch.arange(M, device="cuda") // 128
    x = (s["x_t"].contiguous().view(torch.float8_e4m3fn).double() * s["x_scales"].double()[t].t()).t()
    dx = torch.empty(M, K, dtype=torch.float64, device="cuda")
    dw = torch.empty(G, N, K, dtype=torch.float64, device="cuda")
    for g in range(G):
        at = slice(ends[g], ends[g + 1])
        w = _square64(s["w_t"][:, g * N:(g + 1) * N].t().contiguous(), s["w_scales"][g])
        dx[at] = dy_rows[at] @ w
        dw[g] = dy_columns[at].t() @ x[at]
    return {"dx": dx, "dw": dw}


def _exact_layer(case, s):
    x = s["x"].double()
    logits = x @ s["router"].double().t()
    p = 1 / (1 + torch.exp(-logits)) if case["scoring"] == "sigmoid" else torch.softmax(logits, 1)
    by = p if s["bias"] is None else p + s["bias"].double()
    ids = torch.argsort(by, dim=1, descending=True, stable=True)[:, :case["top"]]
    weights = torch.gather(p, 1, ids)
    weights = weights / weights.sum(1, keepdim=True)
    y = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            h = x[t] @ _square64(s["w13"][e], s["s13"][e]).t()
            gate, up = h[:, :case["I"]], h[:, case["I"]:]
            y[t] += weights[t, j][:, None] * ((gate / (1 + torch.exp(-gate)) * up) @ _square64(s["w2"][e], s["s2"][e]).t())
    return {"y": y, "ids": None, "weights": weights}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("forward", "backward"):
        return _exact_grouped(case, s)
    if case["kind"] == "activations":
        q, d = _quantized64(s["x"], 1)
        q_t, d_t = _quantized64(s["x"], 0)
        return {"q": q, "scales": d.t().contiguous(), "q_t": q_t.t().contiguous(), "scales_t": d_t}
    if case["kind"] == "weights":
        G, N, K = case["groups"], case["N"], case["K"]
        w = s["w"].double().view(G, N, K)
        q = torch.empty_like(w)
        d = torch.empty(G, _ceil(N, 128), _ceil(K, 128), dtype=torch.float64, device="cuda")
        for g in range(G):
            s = _scale64(_block_max64(_block_max64(w[g], 0), 1))
            d[g] = 1.0 / s
            q[g] = _grid64(_held32(w[g] * s.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]))
        q = q.view(G * N, K)
        return {"q": q, "scales": d, "q_t": q.t().contiguous(), "scales_t": None}
    return _exact_layer(case, s)
