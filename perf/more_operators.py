"""Measured cases of what stands around the block-scaled mixture-of-experts layer in a model: the
normalization before it (with the residual's addition and the 8-bit rows that its products read), its
router's balance loss and gradients, and the AdamW step of its weights.

  norm      h = bf16(x + residual), rstd = 1 / sqrt(mean(h^2) + eps), y = h * rstd * w;  8-bit rows of y
            with s = fmax / max(amax, 1e-12) for a row (kept as s) or a block of 1 x 128 (kept as 1 / s)
  router    p = softmax(l) or sigmoid(l) over its sum; loss of a sequence of n tokens
            = experts / (top * n^2) * sum_e count[e] * sum_t p[t, e]; gradients of the logits from the
            losses' and the chosen weights'
  update    m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2,
            p = p - lr * (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + decay * p)
            with m and v in 32 bits, or m and sqrt(v) in e4m3fn with a factor per block of 128: to the
            grid's next value up or down, by a number between 0 and 1 for each element
"""
import math

import numpy as np
import torch

own = False

EPS, BLOCK = 1e-12, 128
NORM_EPS = 1e-6
FMAX = {"fn": 448.0, "fnuz": 240.0}
FP8 = {"fn": torch.float8_e4m3fn, "fnuz": torch.float8_e4m3fnuz}
TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
LR, BETAS, ADAM_EPS, DECAY = 3e-4, (0.9, 0.95), 1e-8, 0.1


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token before the layer: residual and bf16 row, launch latency alone
        {"name": "norm, 1 token", "kind": "norm", "T": 1, "H": 7168, "residual": True, "bf16": True, "scaling": "none", "fmt": "fn", "weight": "bf16"},
        # odd width: rows that start on no boundary, the last block short; one scale a row
        {"name": "norm, odd sizes", "kind": "norm", "T": 1333, "H": 1111, "residual": False, "bf16": False, "scaling": "row", "fmt": "fnuz", "weight": "fp32"},
        # a training batch of a large model: the residual stream, the router's bf16 rows and the products' 8 bits
        {"name": "norm, 16384 tokens", "kind": "norm", "T": 16384, "H": 7168, "residual": True, "bf16": True, "scaling": "block", "fmt": "fn", "weight": "bf16"},
        # gradients in 32 bits (summed over a token's experts), no residual
        {"name": "norm backward, 2048 tokens", "kind": "norm_backward", "T": 2048, "H": 2064, "dh": False, "grad": "fp32", "weight": "fp32"},
        # the backward of that training batch
        {"name": "norm backward, 16384 tokens", "kind": "norm_backward", "T": 16384, "H": 7168, "dh": True, "grad": "bf16", "weight": "bf16"},
        # the smallest layer's router
        {"name": "router, 4 experts", "kind": "router", "T": 96, "E": 4, "top": 2, "S": 1, "scoring": "softmax", "renormalize": True, "logits": "fp32"},
        # fine-grained experts, a balance loss for every one of a batch's ragged sequences
        {"name": "router, 64 experts, 9 sequences", "kind": "router", "T": 8191, "E": 64, "top": 6, "S": 9, "scoring": "softmax", "renormalize": False, "logits": "fp32"},
        # the largest router over a global batch
        {"name": "router, 256 experts", "kind": "router", "T": 65536, "E": 256, "top": 8, "S": 16, "scoring": "sigmoid", "renormalize": True, "logits": "bf16"},
        # the smallest layer's four tensors
        {"name": "update, 4 experts, 8 bits", "kind": "update", "layers": 1, "E": 4, "H": 256, "I": 512, "bits": 8, "param": "bf16", "grad": "bf16"},
        # 24 tensors of odd sizes, 32-bit states and master weights
        {"name": "update, odd sizes, 32 bits", "kind": "update", "layers": 6, "E": 7, "H": 1111, "I": 413, "bits": 32, "param": "master", "grad": "fp32"},
        # a layer of fine-grained experts, states in 8 bits
        {"name": "update, 32 experts, 8 bits", "kind": "update", "layers": 1, "E": 32, "H": 2048, "I": 1408, "bits": 8, "param": "bf16", "grad": "bf16"},
    ]


def _spread(rng, lo, hi):
    return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm_backward", "router", "router", "update"])
    if kind in ("norm", "norm_backward"):
        while True:
            c = {"kind": kind, "T": _spread(rng, 1, 32768), "H": _spread(rng, 64, 8192)}
            if rng.random() < 0.7:  # widths are mostly whole blocks or pieces of 16
                c["H"] = max(64, c["H"] // 16 * 16)
            if c["T"] * c["H"] <= 1.1e8:
                break
        c["weight"] = rng.choice(["bf16", "fp32"])
        if kind == "norm_backward":
            return {**c, "dh": rng.random() < 0.6, "grad": rng.choice(["bf16", "fp32"])}
        scaling = rng.choice(["none", "row", "block", "block"])
        return {**c, "residual": rng.random() < 0.6, "scaling": scaling, "bf16": scaling == "none" or rng.random() < 0.5,
                "fmt": rng.choice(["fn", "fnuz"]) if scaling == "row" else "fn"}
    if kind == "router":
        while True:
            c = {"kind": kind, "T": _spread(rng, 1, 65536), "E": _spread(rng, 2, 512), "top": rng.randint(1, 8), "S": _spread(rng, 1, 64),
                 "scoring": rng.choice(["softmax", "sigmoid"]), "renormalize": rng.random() < 0.6, "logits": rng.choice(["fp32", "bf16"])}
            if c["top"] <= c["E"] and c["T"] * c["E"] <= 1.6e7:
                return c
    while True:
        c = {"kind": kind, "layers": rng.randint(1, 8), "E": _spread(rng, 1, 64), "H": _spread(rng, 64, 4096), "I": _spread(rng, 64, 2048),
             "bits": rng.choice([8, 32]), "param": rng.choice(["bf16", "fp32", "master"]), "grad": rng.choice(["bf16", "fp32"])}
        if 3 * c["layers"] * c["E"] * c["H"] * c["I"] <= (2.5e8 if c["bits"] == 8 else 1e8):
            return c


# ------------------------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(gen, rows, cols):
    """Unit normals with one value in a thousand 30 times as large, as a few channels' are."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x = torch.where(torch.rand(rows, cols, generator=gen, device="cuda") < 1e-3, x * 30, x)
    return x.to(torch.bfloat16)


def _norm_weight(gen, case):
    return (1 + 0.1 * torch.randn(case["H"], generator=gen, device="cuda")).to(TYPE[case["weight"]])


def _ends(seed, rows, count):
    """Ends of count sequences of uneven lengths, one in eight of them empty and, of more than one, a few
    tokens of padding behind the last."""
    rs = np.random.RandomState(seed % (1 << 31))
    p = rs.gamma(2.0, size=count) * (rs.random_sample(count) > 0.125) + 1e-9
    used = rows - (rows // 50 if count > 1 else 0)
    return torch.tensor(np.cumsum(rs.multinomial(used, p / p.sum())), dtype=torch.int32, device="cuda")


def _tensors(case):
    """Sizes of a model's tensors: each layer's norm, router, gate and up, and down weights."""
    E, H, I = case["E"], case["H"], case["I"]
    return [H, E * H, 2 * E * I * H, E * H * I] * case["layers"]


def _places(case):
    """(start, size) of each tensor in a buffer that holds them all, each from a block's start on."""
    sizes = _tensors(case)
    starts = np.cumsum([0] + [_ceil(n, BLOCK) * BLOCK for n in sizes])
    return list(zip(starts[:-1].tolist(), sizes)), int(starts[-1])


def prepare(case, seed):
    gen = _generator(seed)
    kind = case["kind"]
    if kind == "norm":
        s = {"case": case, "x": _activations(gen, case["T"], case["H"]), "w": _norm_weight(gen, case), "residual": None}
        if case["residual"]:
            s["residual"] = _activations(gen, case["T"], case["H"])
        return s
    if kind == "norm_backward":
        h, w = _activations(gen, case["T"], case["H"]), _norm_weight(gen, case)
        g = lambda: (torch.randn(case["T"], case["H"], generator=gen, device="cuda") * 1e-3).to(TYPE[case["grad"]])
        f = h.float()
        return {"case": case, "h": h, "w": w, "rstd": 1 / torch.sqrt((f * f).mean(1) + NORM_EPS), "dy": g(), "dh": g() if case["dh"] else None}
    if kind == "router":
        T, E, S = case["T"], case["E"], case["S"]
        popular = torch.randn(E, generator=gen, device="cuda")  # some experts are asked for more than others
        logits = (torch.randn(T, E, generator=gen, device="cuda") * 1.5 + popular).to(TYPE[case["logits"]])
        ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :case["top"]].to(torch.int32).contiguous()
        return {"case": case, "logits": logits, "ids": ids, "sequences": None if S == 1 else _ends(seed, T, S),
                "dweights": torch.randn(T, case["top"], generator=gen, device="cuda") * 1e-3,
                "dloss": torch.full((S,), 1e-2 / S, device="cuda")}
    # a model some steps into its training, its states as the steps before left them; the seed of a step is its number
    places, total = _places(case)
    flat = lambda scale: torch.randn(total, generator=gen, device="cuda") * scale
    used = torch.cat([torch.nn.functional.pad(torch.ones(n, device="cuda"), (0, -n % BLOCK)) for _, n in places])
    size = torch.exp(flat(1.0)) * 1e-4  # gradients differ in size from element to element
    master, grad = flat(0.02) * used, (flat(1.0) * size * used).to(TYPE[case["grad"]])
    m, r = flat(0.3) * size * used, (0.7 + 0.5 * torch.rand(total, generator=gen, device="cuda")) * size * used
    s = {"case": case, "step": 100, "master": master if case["param"] == "master" else None,
         "param": master.clone() if case["param"] == "fp32" else master.to(torch.bfloat16)}
    if case["bits"] == 8:
        s["m"], s["m_scales"] = _quantize_flat(m, 0.5)
        s["r"], s["r_scales"] = _quantize_flat(r, 0.5)
    else:
        s["m"], s["v"] = m, r * r
    for name, buffer in (("params", s["param"]), ("grads", grad), ("masters", s["master"]), ("ms", s["m"]), ("vs", s.get("v", s.get("r")))):
        s[name] = None if buffer is None else [buffer[at:at + n] for at, n in places]
    for name, buffer in (("m_factors", s.get("m_scales")), ("r_factors", s.get("r_scales"))):
        s[name] = None if buffer is None else [buffer[at // BLOCK:_ceil(at + n, BLOCK)] for at, n in places]
    return s


# ------------------------------------------------------------------------------- plain forms

def _held(y, scale, fmt="fn"):
    return torch.clamp(y * scale, -FMAX[fmt], FMAX[fmt]).to(FP8[fmt])


def _over_amax(amax, fmt="fn"):
    # a quotient of two tensors: a number over a tensor is the number times a rounded reciprocal
    return torch.full_like(amax, FMAX[fmt]) / torch.clamp(amax, min=EPS)


def _plain_norm(s):
    c, out = s["case"], {}
    h = s["x"]
    if s["residual"] is not None:
        h = out["h"] = (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    f = h.float()
    out["rstd"] = 1 / torch.sqrt((f * f).mean(1) + NORM_EPS)
    y = f * out["rstd"][:, None] * s["w"].float()
    if c["bf16"]:
        out["y"] = y.to(torch.bfloat16)
    if c["scaling"] == "row":
        out["scales"] = _over_amax(y.abs().amax(1), c["fmt"])
        out["q"] = _held(y, out["scales"][:, None], c["fmt"])
    if c["scaling"] == "block":
        b = torch.nn.functional.pad(y, (0, -c["H"] % BLOCK)).unflatten(1, (-1, BLOCK))
        scale = _over_amax(b.abs().amax(2))
        out["q"] = _held(b, scale[:, :, None]).flatten(1)[:, :c["H"]].contiguous()
        out["scales"] = (1.0 / scale).t().contiguous()
    return out


def _plain_norm_backward(s):
    x, dy = s["h"].float() * s["rstd"][:, None], s["dy"].float()
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - x * (g * x).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["dy"].dtype), "dw": (dy * x).sum(0)}


def _sequence_of(s):
    """The sequence of each token, S for padding, and the sequences' lengths."""
    c = s["case"]
    if s["sequences"] is None:
        return torch.zeros(c["T"], dtype=torch.long, device="cuda"), torch.tensor([c["T"]], device="cuda")
    ends = s["sequences"].long()
    at = torch.searchsorted(ends, torch.arange(c["T"], device="cuda"), right=True)
    return at, torch.diff(ends, prepend=ends.new_zeros(1))


def _plain_router(s):
    c, l, ids = s["case"], s["logits"].float(), s["ids"].long()
    S, E, top = c["S"], c["E"], c["top"]
    if c["scoring"] == "softmax":
        score = torch.exp(l - l.amax(1, keepdim=True))
        p = score = score / score.sum(1, keepdim=True)
        slope = torch.ones_like(p)  # of log(score) over the logit, before the sum's part
    else:
        score = 1 / (1 + torch.exp(-l))
        p, slope = score / score.sum(1, keepdim=True), 1 - score
    at, length = _sequence_of(s)
    chosen = torch.zeros_like(p).scatter_add_(1, ids, torch.ones_like(s["dweights"]))
    counts = torch.zeros(S + 1, E, device=p.device).index_add_(0, at, chosen)[:S]
    mass = torch.zeros(S + 1, E, device=p.device).index_add_(0, at, p)[:S]
    over = E / (top * torch.clamp(length, min=1).float() ** 2)
    loss = over * (counts * mass).sum(1)
    # gradients: of p from the losses, then of the chosen weights
    dp = torch.nn.functional.pad((s["dloss"] * over)[:, None] * counts, (0, 0, 0, 1))[at]
    dl = p * slope * (dp - (p * dp).sum(1, keepdim=True))
    w = torch.gather(score, 1, ids)
    dw = s["dweights"]
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
        dw = w * (dw - (w * dw).sum(1, keepdim=True))
    elif c["scoring"] == "softmax":
        dl = dl - p * (w * dw).sum(1, keepdim=True)
        dw = w * dw
    else:
        dw = w * dw
    dl.scatter_add_(1, ids, dw * torch.gather(slope, 1, ids))
    return {"loss": loss, "counts": counts.to(torch.int32), "dlogits": dl.to(s["logits"].dtype)}


def _mixed(z):
    """32 bits of z, mixed: two rounds of shift and odd product."""
    z = (z ^ z >> 16) * 0x7F4A7C15 & 0xFFFFFFFF
    z = (z ^ z >> 15) * 0x2C9277B5 & 0xFFFFFFFF
    return z ^ z >> 16


def _random_bits(case, seed):
    """32 random bits for each element: of its tensor's place in the list and of its own place there."""
    places, _ = _places(case)
    keys = [_mixed((seed * 0x9E3779B1 + i) & 0xFFFFFFFF) for i in range(len(places))]
    return torch.cat([_mixed((torch.arange(_ceil(n, BLOCK) * BLOCK, device="cuda") + k) & 0xFFFFFFFF) for (_, n), k in zip(places, keys)])


def _quantize_flat(x, u):
    """Blocks of 128 elements to the grid's value below or above, u in [0, 1) deciding."""
    b = x.view(-1, BLOCK)
    scale = _over_amax(b.abs().amax(1))
    y = torch.clamp(b * scale[:, None], -FMAX["fn"], FMAX["fn"]).flatten()
    step = torch.exp2(torch.clamp(torch.frexp(y)[1] - 1, min=-6).float() - 3)
    q = torch.copysign(torch.floor(y.abs() / step + u) * step, y)
    return q.to(torch.float8_e4m3fn).view(torch.uint8), 1.0 / scale


def _dequantize_flat(q, d):
    return (q.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * d[:, None]).flatten()


def _plain_update(s):
    c, t = s["case"], s["step"]
    places, total = _places(c)
    g = torch.cat([torch.nn.functional.pad(v.float(), (0, -len(v) % BLOCK)) for v in s["grads"]])
    if c["bits"] == 8:
        m, v = _dequantize_flat(s["m"], s["m_scales"]), _dequantize_flat(s["r"], s["r_scales"]).square()
    else:
        m, v = s["m"], s["v"]
    m = BETAS[0] * m + (1 - BETAS[0]) * g
    v = BETAS[1] * v + (1 - BETAS[1]) * g * g
    p = (s["master"] if c["param"] == "master" else s["param"]).float()
    p = p - LR * (m / (1 - BETAS[0] ** t) / (torch.sqrt(v / (1 - BETAS[1] ** t)) + ADAM_EPS) + DECAY * p)
    s["param"].copy_(p)
    if c["param"] == "master":
        s["master"].copy_(p)
    if c["bits"] == 8:
        bits, r = _random_bits(c, t), torch.sqrt(v)
        q, d = _quantize_flat(m, (bits >> 12).float() / 2 ** 20)
        s["m"].copy_(q), s["m_scales"].copy_(d)
        q, d = _quantize_flat(r, ((bits << 16 | bits >> 16) >> 12 & 0xFFFFF).float() / 2 ** 20)
        q = torch.where((r > 0) & (q == 0), torch.ones_like(q), q)  # a nonzero root stays one
        s["r"].copy_(q), s["r_scales"].copy_(d)
    else:
        s["m"].copy_(m), s["v"].copy_(v)


def _updated(s):
    out = {"param": s["param"]}
    if s["case"]["param"] == "master":
        out["master"] = s["master"]
    if s["case"]["bits"] == 32:
        return {**out, "m": s["m"], "v": s["v"]}
    values = lambda q: q.view(torch.float8_e4m3fn)
    return {**out, "m": values(s["m"]), "m_scales": s["m_scales"], "r": values(s["r"]), "r_scales": s["r_scales"]}


# ---------------------------------------------------------------------------------- one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(state, kind)
    if kind == "norm":
        return _plain_norm(state)
    if kind == "norm_backward":
        return _plain_norm_backward(state)
    if kind == "router":
        return _plain_router(state)
    _plain_update(state)
    return _updated(state)


def _own(s, kind):
    import fp8_quantization_grouped_amd as fq
    c = s["case"]
    if kind == "norm":
        fmt = fq.E4M3FN if c["fmt"] == "fn" else fq.E4M3FNUZ
        n = fq.fp8_rms_norm(s["x"], s["w"], NORM_EPS, residual=s["residual"], scaling=None if c["scaling"] == "none" else c["scaling"],
                            fmt=fmt, bf16=c["bf16"])
        out = {"rstd": n.rstd}
        if s["residual"] is not None:
            out["h"] = n.h
        if c["bf16"]:
            out["y"] = n.y
        if c["scaling"] != "none":
            out["q"], out["scales"] = n.q.view(FP8[c["fmt"]]), n.scales
        return out
    if kind == "norm_backward":
        dx, dw = fq.fp8_rms_norm_backward(s["dy"], s["h"], s["rstd"], s["w"], dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if kind == "router":
        loss, counts = fq.moe_balance(s["logits"], s["ids"], scoring=c["scoring"], sequences=s["sequences"])
        dlogits = fq.moe_route_backward(s["logits"], s["ids"], s["dweights"], scoring=c["scoring"], renormalize=c["renormalize"],
                                        dloss=s["dloss"], counts=counts, sequences=s["sequences"])
        return {"loss": loss, "counts": counts, "dlogits": dlogits}
    if "states" not in s:  # kept as long as the parameters are
        if c["bits"] == 8:
            states = {"exp_avg": s["ms"], "exp_avg_sq": s["vs"], "exp_avg_scales": s["m_factors"], "exp_avg_sq_scales": s["r_factors"]}
        else:
            states = {"exp_avg": s["ms"], "exp_avg_sq": s["vs"]}
        s["states"] = fq.AdamWStates(s["params"], bits=c["bits"], masters=s["masters"], **states)
    fq.adamw_step(s["states"], s["grads"], s["step"], LR, betas=BETAS, eps=ADAM_EPS, weight_decay=DECAY)
    return _updated(s)


# -------------------------------------------------------------------------------- their work

def _ceil(a, b):
    return -(-a // b)


def work(case):
    kind = case["kind"]
    if kind == "norm":
        T, H, n = case["T"], case["H"], case["T"] * case["H"]
        wide = 2 + (4 if case["residual"] else 0) + (2 if case["bf16"] else 0) + (0 if case["scaling"] == "none" else 1)
        scales = {"none": 0, "row": 4 * T, "block": 4 * T * _ceil(H, BLOCK)}[case["scaling"]]
        return {"bytes": n * wide + scales + 4 * T + H * (2 if case["weight"] == "bf16" else 4), "flops": 7 * n}
    if kind == "norm_backward":
        T, H, n, g = case["T"], case["H"], case["T"] * case["H"], 2 if case["grad"] == "bf16" else 4
        return {"bytes": n * (2 + 2 * g + (g if case["dh"] else 0)) + 4 * T + H * (6 if case["weight"] == "bf16" else 8), "flops": 10 * n}
    if kind == "router":
        n, one = case["T"] * case["E"], 4 if case["logits"] == "fp32" else 2
        # the losses need every logit before a gradient can be formed, so they are read twice
        return {"bytes": 3 * n * one + 12 * case["T"] * case["top"] + 4 * case["S"] * case["E"], "flops": 20 * n}
    n = sum(_tensors(case))
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    param = {"bf16": 4, "fp32": 8, "master": 10}[case["param"]]
    return {"bytes": int(n * (state + param + (2 if case["grad"] == "bf16" else 4))), "flops": 20 * n}


# --------------------------------------------------------------------------- in 64 bits, apart

def _grid64(v, fmax, emin, u=None):
    """v in 64 bits on the 8-bit grid of three fraction bits: the nearest value (ties to even), or the one below
    or above by u."""
    v = v.clamp(-fmax, fmax)
    e = torch.frexp(v)[1].to(torch.float64) - 1
    step = torch.exp2(e.clamp(min=emin) - 3)
    if u is None:
        return torch.round(v / step) * step
    return torch.sign(v) * torch.floor(v.abs() / step + u) * step


def _exact_norm(case, s):
    out = {}
    h = s["x"].double()
    if case["residual"]:
        h = h + s["residual"].double()
        out["h"] = h
        h = h.to(torch.bfloat16).double()  # the residual stream is held in bf16, and the norm is of that
    var = h.square().sum(1) / case["H"]
    out["rstd"] = (var + NORM_EPS) ** -0.5
    y = h * out["rstd"].unsqueeze(1) * s["w"].double()
    if case["bf16"]:
        out["y"] = y
    if case["scaling"] == "none":
        return out
    fmax, emin = (448.0, -6) if case["fmt"] == "fn" else (240.0, -7)
    width = case["H"] if case["scaling"] == "row" else 128
    at = torch.arange(case["H"], device="cuda") // width
    top = torch.zeros(case["T"], int(at[-1]) + 1, dtype=torch.float64, device="cuda").scatter_reduce(1, at.expand_as(y), y.abs(), "amax")
    scale = fmax / top.clamp(min=1e-12)
    out["q"] = _grid64(y * scale[:, at], fmax, emin)
    out["scales"] = scale[:, 0] if case["scaling"] == "row" else (1 / scale).t().contiguous()
    return out


def _exact_norm_backward(case, s):
    h, r, w, dy = (s[k].double() for k in ("h", "rstd", "w", "dy"))
    inner = torch.matmul(h * dy, w) / case["H"]
    dx = r[:, None] * (dy * w) - (r ** 3 * inner)[:, None] * h
    if case["dh"]:
        dx += s["dh"].double()
    return {"dx": dx, "dw": torch.matmul(r, dy * h)}


def _exact_router(case, s):
    """By one sequence after the other, the gradient by the chain of derivatives of log p."""
    T, E, S, top = case["T"], case["E"], case["S"], case["top"]
    l, ids = s["logits"].double(), s["ids"].long()
    soft = case["scoring"] == "softmax"
    score = torch.softmax(l, 1) if soft else torch.sigmoid(l)
    p = score / score.sum(1, keepdim=True)
    ends = [0] + ([T] if s["sequences"] is None else s["sequences"].tolist())
    loss, dl = torch.zeros(S, dtype=torch.float64, device="cuda"), torch.zeros(T, E, dtype=torch.float64, device="cuda")
    for i in range(S):
        a, b = ends[i], ends[i + 1]
        if b > a:
            f = torch.bincount(ids[a:b].flatten(), minlength=E).double() * E / (top * (b - a))
            loss[i] = f @ p[a:b].mean(0)
            g = s["dloss"][i].double() * f / (b - a)
            dl[a:b] = p[a:b] * (g - (p[a:b] @ g)[:, None])
    if not soft:
        dl = dl * (1 - score)
    w, dw = torch.gather(score, 1, ids), s["dweights"].double()
    total = w.sum(1, keepdim=True)
    dscore = (dw - (dw * w).sum(1, keepdim=True) / total) / total if case["renormalize"] else dw
    ds = torch.zeros_like(dl).scatter_add_(1, ids, dscore)
    dl += score * (ds - (ds * score).sum(1, keepdim=True)) if soft else ds * score * (1 - score)
    return {"loss": loss, "counts": None, "dlogits": dl}


def _exact_update(case, s):
    places, total = _places(case)
    t = s["step"]
    spread = lambda d: d.double().repeat_interleave(128)
    eight = case["bits"] == 8
    if eight:
        m = s["m"].view(torch.float8_e4m3fn).double() * spread(s["m_scales"])
        v = (s["r"].view(torch.float8_e4m3fn).double() * spread(s["r_scales"])) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    for (at, n), g in zip(places, s["grads"]):
        m[at:at + n] = BETAS[0] * m[at:at + n] + (1 - BETAS[0]) * g.double()
        v[at:at + n] = BETAS[1] * v[at:at + n] + (1 - BETAS[1]) * g.double() ** 2
    p = s["master" if case["param"] == "master" else "param"].double()
    p = p * (1 - LR * DECAY) - LR * (m / (1 - BETAS[0] ** t)) / ((v / (1 - BETAS[1] ** t)).sqrt() + ADAM_EPS)
    out = {"param": p}
    if case["param"] == "master":
        out["master"] = p
    if not eight:
        return {**out, "m": m, "v": v}
    word = torch.cat([torch.arange(-(-n // 128) * 128, device="cuda") + _key64(t, i) for i, (_, n) in enumerate(places)]) % 2 ** 32
    word = _word64(word)
    for name, x, u in (("m", m, word // 2 ** 12), ("r", v.sqrt(), word % 2 ** 16 * 2 ** 4 + word // 2 ** 28)):
        scale = 448.0 / x.abs().view(-1, 128).amax(1).clamp(min=1e-12)
        q = _grid64(x * scale.repeat_interleave(128), 448.0, -6, u.double() / 2 ** 20)
        out[name] = torch.where((x > 0) & (q == 0), 2.0 ** -9, q) if name == "r" else q
        out[name + "_scales"] = 1 / scale
    return out


def _word64(z):
    z = z.bitwise_xor(z // 2 ** 16) * 2135587861 % 2 ** 32
    z = z.bitwise_xor(z // 2 ** 15) * 747796405 % 2 ** 32
    return z.bitwise_xor(z // 2 ** 16)


def _key64(seed, i):
    return int(_word64(torch.tensor([(seed * 2654435761 + i) % 2 ** 32]))[0])


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "router": _exact_router, "update": _exact_update}[case["kind"]](case, s)
