"""Routing and the mixture-of-experts layer for a few tokens, against 64-bit arithmetic."""
from __future__ import annotations

import pytest
import torch

from tests import blocklib as bl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_quantization_grouped_amd as m
    m.lib()
    return m


def normal(seed, *shape, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16).to(DEV)


# ---------------------------------------------------------------------------------------- routing

def plain_route(x, router, k, bias, scoring, renorm, scale):
    logits = x.cpu().double() @ router.cpu().double().t()
    p = torch.sigmoid(logits) if scoring == "sigmoid" else torch.softmax(logits, 1)
    by = logits if bias is None else p + bias.cpu().double()
    ids = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(p, 1, ids)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    return logits, by, ids, w * scale


@pytest.mark.parametrize("scoring,with_bias,renorm,scale", [("softmax", False, True, 1.0), ("softmax", False, False, 1.0),
                                                             ("sigmoid", True, True, 2.5), ("sigmoid", False, False, 1.0), ("softmax", True, True, 1.0)])
@pytest.mark.parametrize("T,H,E,k", [(1, 8, 1, 1), (1, 7168, 32, 8), (3, 136, 5, 5), (17, 2048, 64, 6), (64, 264, 65, 8),
                                     (130, 512, 256, 8), (5, 1024, 1000, 32), (33, 40, 300, 3)])
def test_route(fq, T, H, E, k, scoring, with_bias, renorm, scale):
    x, r = normal(T + H, T, H), normal(E, E, H, scale=H ** -0.5)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(1)).to(DEV) * 0.2 if with_bias else None
    ids, w = fq.moe_route(x, r, k, bias=bias, scoring=scoring, renormalize=renorm, scale=scale)
    logits, by, want, want_w = plain_route(x, r, k, bias, scoring, renorm, scale)
    got = ids.cpu().long()
    assert got.shape == (T, k) and bool((got >= 0).all()) and bool((got < E).all())
    assert all(len(set(row)) == k for row in got.tolist())
    # an fp32 sum of H terms is off by at most H 2^-24 of their magnitudes' sum; scores no more
    tol = H * 2.0 ** -24 * (x.cpu().double().abs() @ r.cpu().double().abs().t()).amax(1, keepdim=True) + 2.0 ** -21
    chosen = torch.gather(by, 1, got)
    best = torch.gather(by, 1, want)
    assert bool(((chosen - best).abs() <= 2 * tol).all())  # the same values in the same order
    exact_w = torch.gather(torch.sigmoid(logits) if scoring == "sigmoid" else torch.softmax(logits, 1), 1, got)
    if renorm:
        exact_w = exact_w / exact_w.sum(1, keepdim=True)
    # relative error of a score: that of its logit's exponential, twice with the sum's, and roundings
    assert bool(((w.cpu().double() - exact_w * scale).abs() <= (4 * tol + 2.0 ** -19) * exact_w * scale).all())


def test_route_ties_go_to_the_lowest_index(fq):
    x = torch.ones(3, 64, dtype=torch.bfloat16, device=DEV)
    r = torch.zeros(100, 64, dtype=torch.bfloat16, device=DEV)
    r[70] = r[20] = r[21] = 0.5
    for scoring, bias in (("softmax", None), ("sigmoid", None), ("sigmoid", torch.zeros(100, device=DEV))):
        ids, w = fq.moe_route(x, r, 6, bias=bias, scoring=scoring)
        assert ids.tolist() == [[20, 21, 70, 0, 1, 2]] * 3
    ids, _ = fq.moe_route(x, r, 4, bias=torch.full((100,), float("-inf"), device=DEV))
    assert ids.tolist() == [[0, 1, 2, 3]] * 3
    bias = torch.zeros(100, device=DEV)
    bias[5] = 10
    ids, w = fq.moe_route(x, r, 2, bias=bias, scoring="sigmoid", renormalize=False)
    assert ids.tolist() == [[5, 20]] * 3 and abs(float(w[0, 0]) - 0.5) < 1e-6  # the bias is no weight


def test_route_with_nan_still_names_experts(fq):
    x, r = normal(1, 4, 128), normal(2, 40, 128, scale=0.1)
    clean, _ = fq.moe_route(x, r, 4)
    r[7] = float("nan")
    x[2] = float("nan")
    ids, w = fq.moe_route(x, r, 4)
    assert ids[2].tolist() == [0, 1, 2, 3]
    for t in (0, 1, 3):
        assert 7 not in ids[t].tolist()
        assert [e for e in clean[t].tolist() if e != 7][:3] == ids[t].tolist()[:3]


# ------------------------------------------------------------------------------------------ layer

def layer(fq, seed, E, H, I):
    w13, w2 = normal(seed, E * 2 * I, H, scale=0.05), normal(seed + 1, E * H, I, scale=0.05)
    q13, _, s13 = fq.fp8_block_quant_weights(w13, E)
    q2, _, s2 = fq.fp8_block_quant_weights(w2, E)
    return q13.unflatten(0, (E, 2 * I)), s13, q2.unflatten(0, (E, H)), s2


def check_layer(y, x, ids, weights, w13, s13, w2, s2):
    """y against the formula, with a bound from the roundings: sums of up to 7168 products in 32 bits
    (chains of at most about 2^8 additions: 2^-16 of the magnitudes), h and y rounded to bf16."""
    T, H = x.shape
    E, I = w2.shape[0], w2.shape[2]
    xs = x.cpu().double()
    want = torch.zeros(T, H, dtype=torch.float64)
    tol = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            a = bl.real_square(w13[e], s13[e])
            b = bl.real_square(w2[e], s2[e])
            gu, mags = a @ xs[t], a.abs() @ xs[t].abs()
            g, u = gu[:I], gu[I:]
            act = g * torch.sigmoid(g)
            h = act * u
            off = 2.0 ** -16 * (1.1 * mags[:I] * u.abs() + act.abs() * mags[I:]) + (2.0 ** -8 + 2.0 ** -20) * h.abs()
            w = float(weights[t, j])
            want[t] += w * (b @ h)
            tol[t] += abs(w) * (b.abs() @ off + 2.0 ** -16 * (b.abs() @ h.abs()))
    got = y.cpu().double()
    assert bool(torch.isfinite(got).all())
    over = (got - want).abs() - tol - 2.0 ** -8 * want.abs() - 1e-30
    assert float(over.max()) <= 0
    if float(want.norm()) > 0:  # the roundings are independent: their norm is far below their sum
        assert float((got - want).norm() / want.norm()) < 2.0 ** -8


LAYERS = [  # T, H, I, E, k
    (1, 16, 16, 1, 1), (1, 128, 128, 4, 2), (2, 256, 512, 4, 2), (1, 512, 256, 40, 8), (5, 144, 176, 7, 3), (16, 272, 96, 5, 5),
    (17, 256, 144, 3, 2), (40, 128, 128, 2, 2), (64, 400, 208, 9, 4), (65, 128, 64, 4, 3), (128, 96, 32, 3, 1), (3, 2064, 48, 300, 2),
    (7, 48, 2064, 6, 6)]


@pytest.mark.parametrize("T,H,I,E,k", LAYERS)
def test_layer(fq, T, H, I, E, k):
    x, r = normal(T, T, H), normal(E, E, H, scale=H ** -0.5)
    w = layer(fq, H + I, E, H, I)
    ids, weights = fq.moe_route(x, r, k)
    y = fq.fp8_moe_few_tokens(x, ids, weights, *w)
    check_layer(y, x, ids, weights, *w)
    assert torch.equal(y, fq.fp8_moe_few_tokens(x, ids, weights, *w))  # the same sums every time


@pytest.mark.parametrize("T,E", [(4, 3), (20, 4), (100, 2), (2, 60)])
def test_all_tokens_to_one_expert_and_ids_outside(fq, T, E):
    """One expert takes every token (several token tiles), others none; ids outside add nothing and
    a token without experts gives zeros; a token may name an expert twice."""
    H, I, k = 144, 80, 3
    x = normal(T, T, H)
    w = layer(fq, 3, E, H, I)
    ids = torch.full((T, k), E - 1, dtype=torch.int32, device=DEV)
    ids[:, 0] = -1
    ids[:, 2] = E
    ids[0] = torch.tensor([E + 5, -7, 2 ** 31 - 1])
    ids[T - 1] = torch.tensor([E - 1, E - 1, 0])
    weights = torch.rand(T, k, generator=torch.Generator().manual_seed(T)).to(DEV)
    y = fq.fp8_moe_few_tokens(x, ids, weights, *w)
    check_layer(y, x, ids, weights, *w)
    assert not bool(y[0].any())


def test_every_weight_code(fq):
    """Each finite e4m3fn code reaches the product with its value: identity-like experts."""
    H, I, E = 256, 256, 1
    codes = torch.arange(256, dtype=torch.uint8)
    codes = torch.where((codes & 0x7F) == 0x7F, torch.zeros_like(codes), codes)
    w13 = torch.zeros(1, 2 * I, H, dtype=torch.uint8)
    w13[0, :I, 0] = 0x38              # gate rows: 1 at column 0
    w13[0, I:, 1] = codes             # up row i: code i at column 1
    w2 = torch.zeros(1, H, I, dtype=torch.uint8)
    w2[0, range(H), range(H)] = 0x38  # identity
    one = lambda n: torch.ones(1, -(-n // 128), 2, device=DEV)
    x = torch.zeros(1, H, dtype=torch.bfloat16, device=DEV)
    x[0, 0], x[0, 1] = 64.0, 1.0      # silu(64) = 64 in 32 bits
    ids = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    y = fq.fp8_moe_few_tokens(x, ids, torch.ones(1, 1, device=DEV), w13.to(DEV), one(2 * I), w2.to(DEV), one(H))
    assert torch.equal(y.cpu().double()[0], 64.0 * bl.decode(codes))


def test_rows_do_not_meet(fq):
    """A token of infinities and NaN leaves the others' results as they are."""
    x = normal(1, 9, 256)
    w = layer(fq, 2, 3, 256, 128)
    ids = torch.tensor([[t % 3, (t + 1) % 3] for t in range(9)], dtype=torch.int32, device=DEV)
    weights = torch.full((9, 2), 0.5, device=DEV)
    clean = fq.fp8_moe_few_tokens(x, ids, weights, *w)
    x2 = x.clone()
    x2[4] = float("nan")
    x2[7] = float("inf")
    y = fq.fp8_moe_few_tokens(x2, ids, weights, *w)
    keep = [t for t in range(9) if t not in (4, 7)]
    assert torch.equal(y[keep], clean[keep]) and bool(y[4].isnan().all())


def test_strided_operands_and_transposed_weight_storage(fq):
    """x and y inside larger buffers; weights side by side in one [n, E * k] matrix."""
    T, H, I, E = 6, 256, 160, 4
    w13, s13, w2, s2 = layer(fq, 5, E, H, I)
    x = normal(3, T, H)
    wide = torch.full((T, H + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :H] = x
    ids, weights = fq.moe_route(x, normal(4, E, H, scale=0.1), 2)
    want = fq.fp8_moe_few_tokens(x, ids, weights, w13, s13, w2, s2)
    beside = lambda w: w.transpose(0, 1).contiguous().view(w.shape[1], -1).unflatten(1, (E, w.shape[2])).transpose(0, 1)
    y = torch.full((T, H + 3), 9.0, dtype=torch.bfloat16, device=DEV)
    fq.fp8_moe_few_tokens(wide[:, :H], ids, weights, beside(w13), s13.transpose(1, 2).contiguous().transpose(1, 2),
                          beside(w2.view(torch.float8_e4m3fn)), s2, y=y[:, :H])
    assert torch.equal(y[:, :H], want) and bool((y[:, H:] == 9).all())


def test_graph_and_other_stream(fq):
    T, H, I, E = 3, 256, 256, 8
    w = layer(fq, 5, E, H, I)
    r = normal(4, E, H, scale=0.1)
    xs = [normal(s, T, H) for s in range(4)]

    def step(x):
        ids, weights = fq.moe_route(x, r, 2, scoring="sigmoid")
        return fq.fp8_moe_few_tokens(x, ids, weights, *w)

    want = [step(x) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(xs[1])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[1])
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step(x)
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        assert torch.equal(step(xs[(i + 1) % 4]), want[(i + 1) % 4])


def test_agrees_with_the_grouped_products(fq):
    """The same layer through the block-scaled grouped products: they quantize the activations, so
    the two differ by that rounding (2^-4 relative per element, averaged over the contraction)."""
    T, H, I, E, k = 32, 512, 256, 4, 2
    x = normal(1, T, H)
    w13, s13, w2, s2 = layer(fq, 7, E, H, I)
    ids, weights = fq.moe_route(x, normal(2, E, H, scale=0.05), k)
    y = fq.fp8_moe_few_tokens(x, ids, weights, w13, s13, w2, s2)
    flat = ids.flatten().long()
    order = torch.argsort(flat, stable=True)
    off = torch.cumsum(torch.bincount(flat, minlength=E), 0).to(torch.int32)
    F = fq.GEMM_FWD_MGROUPED
    h = fq.fp8_block_grouped_gemm(F, *fq.fp8_block_quant_rowwise(x[order // k]), w13, s13, off).float()
    h = (torch.nn.functional.silu(h[:, :I]) * h[:, I:]).to(torch.bfloat16)
    o = fq.fp8_block_grouped_gemm(F, *fq.fp8_block_quant_rowwise(h), w2, s2, off).float()
    out = torch.zeros(T, H, device=DEV).index_add_(0, order // k, o * weights.flatten()[order][:, None])
    assert float((y.float() - out).norm() / out.norm()) < 2.0 ** -4


def test_refusals(fq):
    T, H, I, E = 4, 64, 32, 3
    x, r = normal(1, T, H), normal(2, E, H)
    w13, s13, w2, s2 = layer(fq, 3, E, H, I)
    ids, weights = fq.moe_route(x, r, 2)
    L = fq.fp8_moe_few_tokens
    for bad in (lambda: fq.moe_route(x.float(), r, 2), lambda: fq.moe_route(x, r, 0), lambda: fq.moe_route(x, r, 4),
                lambda: fq.moe_route(x, r[:, :32], 2), lambda: fq.moe_route(x, r, 2, scoring="tanh"), lambda: fq.moe_route(x, r, 2, bias=torch.zeros(2, device=DEV)),
                lambda: fq.moe_route(x, r.cpu(), 2), lambda: L(x, ids.long(), weights, w13, s13, w2, s2), lambda: L(x, ids[:2], weights, w13, s13, w2, s2),
                lambda: L(x, ids, weights[:, :1], w13, s13, w2, s2), lambda: L(x, ids, weights, w13[:, :62], s13, w2, s2),
                lambda: L(x, ids, weights, w13, s13[:2], w2, s2), lambda: L(x, ids, weights, w13, s13, w2[:2], s2),
                lambda: L(x, ids, weights, w13, s13, w2, s2.double()), lambda: L(x, ids, weights, w13, s13, w2, s2, y=torch.empty(T, H, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    big = normal(1, 129, H)
    i2, g2 = fq.moe_route(big, r, 2)
    with pytest.raises(RuntimeError, match="unsupported"):
        L(big, i2, g2, w13, s13, w2, s2)
    with pytest.raises(RuntimeError, match="workspace"):
        L(x, ids, weights, w13, s13, w2, s2, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


def test_no_tokens(fq):
    H, I, E = 64, 32, 3
    x = torch.empty(0, H, dtype=torch.bfloat16, device=DEV)
    ids, weights = fq.moe_route(x, normal(2, E, H), 2)
    assert ids.shape == (0, 2)
    assert fq.fp8_moe_few_tokens(x, ids, weights, *layer(fq, 3, E, H, I)).shape == (0, H)


def test_experts_past_32_bits(fq):
    """The last experts' weights start past 4 GiB."""
    T, H, I, E = 3, 4096, 2048, 300  # w13: 300 x 16 MiB
    w13 = torch.randint(0, 120, (E, 2 * I, H), dtype=torch.uint8, device=DEV)
    s13 = torch.rand(E, 2 * I // 128, H // 128, device=DEV) * 1e-4
    w2 = torch.randint(0, 120, (E, H, I), dtype=torch.uint8, device=DEV)
    s2 = torch.rand(E, H // 128, I // 128, device=DEV) * 1e-3
    x = normal(1, T, H)
    ids = torch.tensor([[E - 1, E - 2]] * T, dtype=torch.int32, device=DEV)
    weights = torch.full((T, 2), 0.5, device=DEV)
    y = fq.fp8_moe_few_tokens(x, ids, weights, w13, s13, w2, s2)
    want = fq.fp8_moe_few_tokens(x, ids - (E - 2), weights, w13[-2:].clone(), s13[-2:].clone(), w2[-2:].clone(), s2[-2:].clone())
    assert torch.equal(y, want) and bool(y.isfinite().all()) and bool(y.any())


@pytest.mark.parametrize("T,H,I,E,k", [(34, 400, 1040, 6, 2), (100, 512, 528, 3, 2), (128, 1040, 400, 4, 4), (70, 2048, 272, 2, 1)])
def test_many_tokens_of_few_experts(fq, T, H, I, E, k):
    """Several passes of 32 tokens over an expert's weights, the contraction in parts."""
    x = normal(T + 1, T, H)
    w = layer(fq, H + I, E, H, I)
    g = torch.Generator().manual_seed(T)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).to(DEV)
    ids[: T // 2, 0] = E - 1  # the last expert takes more than half of the tokens
    weights = torch.rand(T, k, generator=g).to(DEV)
    y = fq.fp8_moe_few_tokens(x, ids, weights, *w)
    check_layer(y, x, ids, weights, *w)
    for t in (0, T - 1):  # and tokens by themselves
        one = fq.fp8_moe_few_tokens(x[t:t + 1], ids[t:t + 1], weights[t:t + 1], *w)
        check_layer(one, x[t:t + 1], ids[t:t + 1], weights[t:t + 1], *w)
