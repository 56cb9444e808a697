"""adamw_step against 64 bits (tests/adamlib.py)."""
from __future__ import annotations

import pytest
import torch

from tests import adamlib as al

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
SIZES = [1, 7, 8, 127, 128, 129, 1000, 2047, 2048, 2049, 4096, 5000, 100003]


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_quantization_grouped_amd as m
    m.lib()
    return m


def normal(n, seed, dtype=F32, scale=1.0, shift=0):
    """n normals, shift elements behind an allocation's start."""
    x = torch.randn(n, generator=torch.Generator().manual_seed(seed)) * scale
    return torch.cat([torch.zeros(shift), x]).to(dtype).cuda()[shift:]


def states_of(fq, params, bits, masters=None, seed=0):
    """States as some steps leave them."""
    if bits == 32:
        m = [normal(p.numel(), seed + i, scale=1e-3).view(p.shape) for i, p in enumerate(params)]
        return fq.AdamWStates(params, 32, masters, m, [(x * 3).square() + 1e-9 for x in m])
    kept = [[], [], [], []]
    for i, p in enumerate(params):
        n = p.numel()
        for at, x in ((0, normal(n, seed + i, BF16, 1e-3)), (1, (normal(n, seed + i + 50, BF16, 3e-3).abs() + 1e-4).to(BF16))):
            q, d = fq.fp8_block_quant_rowwise(x[None])
            kept[at].append(q[0].contiguous())
            kept[at + 2].append(d[:, 0].contiguous())
    return fq.AdamWStates(params, 8, masters, *kept)


def values(s):
    """Copies of (parameters or masters, first moments, second moments) in 64 bits."""
    p = [(m if m is not None else p).cpu().double().flatten() for p, m in zip(s.params, s.masters)]
    if s.bits == 32:
        return p, [m.cpu().double().flatten() for m in s.exp_avg], [v.cpu().double().flatten() for v in s.exp_avg_sq]
    return (p, [al.decode(*t) for t in zip(s.exp_avg, s.exp_avg_scales)],
            [al.decode(*t).square() for t in zip(s.exp_avg_sq, s.exp_avg_sq_scales)])


def check(s, before, grads, t, lr, betas, eps, decay, seed=0, scale=1.0):
    for i, g in enumerate(grads):
        p, m, v = (b[i] for b in before)
        n = len(p)
        if g is None or n == 0:
            continue
        p1, off_p, m1, off_m, v1, off_v = al.step64(p, g.cpu().double().flatten(), m, v, t, lr, betas, eps, decay, scale)
        half = al.U if s.params[i].dtype is F32 else 2.0 ** -8
        got = s.params[i].cpu().double().flatten()
        assert bool(((got - p1).abs() <= (1 + half) * off_p + half * p1.abs()).all()), i
        if s.masters[i] is not None:
            master = s.masters[i].cpu().flatten()
            assert bool(((master.double() - p1).abs() <= off_p).all())
            assert torch.equal(s.params[i].cpu().flatten(), master.to(BF16))
        if s.bits == 32:
            assert bool(((s.exp_avg[i].cpu().double().flatten() - m1).abs() <= off_m).all())
            assert bool(((s.exp_avg_sq[i].cpu().double().flatten() - v1).abs() <= off_v).all())
        else:
            w = al.words(seed + t, i, n)
            al.check_kept(s.exp_avg[i], s.exp_avg_scales[i], m1, off_m, w, False)
            # v known up to off_v, its root lies between those of v - off_v and v + off_v: for squares below
            # 32 bits' normal range that is all of it
            r = torch.sqrt(v1)
            off_r = torch.maximum(torch.sqrt(v1 + off_v) - r, r - torch.sqrt((v1 - off_v).clamp(min=0))) + 2 * al.U * r
            al.check_kept(s.exp_avg_sq[i], s.exp_avg_sq_scales[i], r, off_r, w, True)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("param", ["bf16", "fp32", "master"])
@pytest.mark.parametrize("grad", [BF16, F32])
def test_step(fq, bits, param, grad):
    masters = [normal(n, i) for i, n in enumerate(SIZES)] if param == "master" else None
    params = [m.to(BF16) for m in masters] if masters else [normal(n, i, BF16 if param == "bf16" else F32) for i, n in enumerate(SIZES)]
    s = states_of(fq, params, bits, masters)
    grads = [normal(n, 100 + i, grad, 2e-3) for i, n in enumerate(SIZES)]
    for t in (5, 6):
        before = values(s)
        fq.adamw_step(s, grads, t, 1e-2, betas=(0.9, 0.95), weight_decay=0.1)
        check(s, before, grads, t, 1e-2, (0.9, 0.95), 1e-8, 0.1)


@pytest.mark.parametrize("bits", [8, 32])
def test_first_step_from_zeros(fq, bits):
    params = [normal(3000, 1).view(30, 100), normal(300, 2, BF16)]
    s = fq.AdamWStates(params, bits)
    grads = [normal(3000, 3, scale=1e-4).view(30, 100), normal(300, 4, scale=1e-20)]  # squares that vanish
    before = values(s)
    fq.adamw_step(s, grads, 1, 1e-3, betas=(0.9, 0.999), seed=77)
    check(s, before, grads, 1, 1e-3, (0.9, 0.999), 1e-8, 0.01, seed=77)


@pytest.mark.parametrize("bits", [8, 32])
def test_many_tensors_of_all_kinds(fq, bits):
    """More than a launch takes, types mixed, some without gradient, some empty, some that start on no boundary."""
    params, masters, grads = [], [], []
    for i in range(100):
        n = [0, 1, 130, 2048, 777, 3000, 64][i % 7]
        shift = [0, 1, 4][i % 3]
        params.append(normal(n, i, BF16 if i % 2 else F32, shift=shift))
        masters.append(params[-1].float() if i % 4 == 1 else None)
        grads.append(None if i % 11 == 5 else normal(n, 200 + i, F32 if i % 5 else BF16, 1e-2, shift=shift))
    s = states_of(fq, params, bits, masters)
    keep = [[None if t is None else t.clone() for t in group] for group in (params, s.masters, s.exp_avg, s.exp_avg_sq)]
    before = values(s)
    fq.adamw_step(s, grads, 10, 1e-2, seed=3)
    check(s, before, grads, 10, 1e-2, (0.9, 0.999), 1e-8, 0.01, seed=3)
    for i, g in enumerate(grads):
        if g is None:
            for kept, now in zip(keep, (params, s.masters, s.exp_avg, s.exp_avg_sq)):
                assert kept[i] is None or torch.equal(kept[i], now[i])


def test_memory_around_the_tensors_is_left(fq):
    for bits in (8, 32):
        buffers = [torch.full((700,), 7, dtype=d, device="cuda") for d in ((BF16, F32, torch.uint8, torch.uint8, F32, F32) if bits == 8 else (BF16, F32, F32, F32))]
        cut = [b[131:131 + 303] for b in buffers[:4]] + [b[131:134] for b in buffers[4:]]
        for c in cut:
            c.zero_()
        s = fq.AdamWStates(cut[:1], bits, cut[1:2], *[[c] for c in cut[2:]])
        fq.adamw_step(s, [normal(303, 1, BF16)], 1, 1e-2)
        for b, c in zip(buffers, cut):
            assert bool((b[:131] == 7).all()) and bool((b[131 + len(c):] == 7).all()) and bool((c != 0).any())


def test_steps_repeat_to_the_bit_and_seeds_differ(fq):
    def after(seed, t=4):
        p = [normal(5000, 1, BF16)]
        s = states_of(fq, p, 8)
        fq.adamw_step(s, [normal(5000, 2, BF16, 1e-2)], t, 1e-3, seed=seed)
        return torch.cat([s.exp_avg[0], s.exp_avg_sq[0]]), p[0]

    a, b, c, d = after(0), after(0), after(1), after(1, 3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert not torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])  # the step itself takes no random bits
    assert float((a[0] != c[0]).float().mean()) > 0.2


def test_kept_states_are_unbiased(fq):
    """The mean over many elements of one value: its rounding's deviation is at most half a step each."""
    n = 1 << 18
    p = [torch.zeros(n, device="cuda")]
    g = torch.full((n,), 0.777, device="cuda")
    g[::128] = 1.0  # every block's largest
    s = fq.AdamWStates(p, 8)
    fq.adamw_step(s, [g], 1, 1e-3)
    m, v = values(s)[1:]
    rest = torch.ones(n, dtype=torch.bool)
    rest[::128] = False
    for got, want in ((m[0][rest], 0.1 * 0.777), (v[0].sqrt()[rest], 0.001 ** 0.5 * 0.777)):
        steps = want * 2.0 ** -3  # of the grid, at most
        assert 2 <= len(got.unique()) <= 4  # the values on both sides (their factors may differ in the last bit)
        assert abs(float(got.mean()) - want) <= 6 * steps / 2 / len(got) ** 0.5 + 1e-6 * want


@pytest.mark.parametrize("beta2", [0.95, 0.999])
def test_long_averages_follow_their_gradients(fq, beta2):
    """One step changes r by as little as a 2000th of itself, far below the grid's steps: it moves all the same.
    A value on the grid that moves by e of itself falls f = e / step between two of them and is rounded with
    a variance of f (1 - f) step^2 <= e step; over the 1 / (1 - beta2) steps that the average remembers, each
    changing r by up to (1 - beta2) / 2 of itself, these add to step / 2 <= 2^-4 of r^2: a spread of 0.25 at
    most, half its square of which is the mean root's distance from the root of the mean square."""
    n = 1 << 14
    g = normal(n, 1).exp()
    s = fq.AdamWStates([torch.zeros(n, device="cuda")], 8)
    for t in range(1, 701):
        fq.adamw_step(s, [g], t, 0.0, betas=(0.9, beta2))
    m, v = values(s)[1:]
    size = g.cpu().double()
    for got, want in ((m[0], size), (v[0].sqrt(), size * (1 - beta2 ** 700) ** 0.5)):
        q = got / want
        assert abs(float(q.mean()) - 1) <= 0.25 ** 2 / 2 + 6 * 0.25 / n ** 0.5
        assert float((q - 1).square().mean()) <= 0.25 ** 2


@pytest.mark.parametrize("bits", [8, 32])
def test_device_step_rate_and_scale(fq, bits):
    p = [normal(3000, 1), normal(500, 2, BF16)]
    s = states_of(fq, p, bits)
    grads = [normal(3000, 3, scale=1e-2), normal(500, 4, BF16, 1e-2)]
    for t in (1, 2, 1000, 1 << 30):
        before = values(s)
        fq.adamw_step(s, grads, torch.tensor([t], dtype=torch.int32, device="cuda"), torch.tensor(2e-3, device="cuda"), seed=9,
                      grad_scale=torch.tensor([0.25], device="cuda"))
        check(s, before, grads, t, 2e-3, (0.9, 0.999), 1e-8, 0.01, seed=9, scale=0.25)


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_step(fq, bits):
    """Replays with the step and rate of the device, against the same steps made eagerly."""
    def fresh():
        p = [normal(3000, 1, BF16), normal(700, 2)]
        return states_of(fq, p, bits), [normal(3000, 3, BF16, 1e-2), normal(700, 4, scale=1e-2)]

    (a, ga), (b, gb) = fresh(), fresh()
    step, lr = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fq.adamw_step(a, ga, step, lr)
    for t in range(1, 5):
        step.fill_(t)
        lr.fill_(1e-2 / t)
        for x, y in zip(ga, gb):
            x.normal_(generator=torch.Generator("cuda").manual_seed(t))
            y.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        fq.adamw_step(b, gb, step, lr)
        for x, y in zip(a.params + a.exp_avg + a.exp_avg_sq, b.params + b.exp_avg + b.exp_avg_sq):
            assert torch.equal(x, y), t


def test_states_go_into_the_block_format(fq):
    """The first moments' bytes and factors are those of one row of fp8_block_quant_rowwise wherever the
    values are on the grid."""
    n = 1000
    x = torch.exp2(torch.randint(-3, 4, (n,), generator=torch.Generator().manual_seed(1)).float()).cuda()
    x[::128] = 448.0
    s = fq.AdamWStates([torch.zeros(n, device="cuda")], 8)
    fq.adamw_step(s, [x], 1, 1e-3, betas=(0.0, 0.5))
    q, d = fq.fp8_block_quant_rowwise(x.to(BF16)[None])
    assert torch.equal(s.exp_avg[0], q[0]) and torch.equal(s.exp_avg_scales[0], d[:, 0])


@pytest.mark.parametrize("bits,n", [(32, 6_000_077), (8, 14_000_077)])
def test_steps_past_the_caches(fq, bits, n):
    """More than the last-level cache holds, where reads and writes go past the caches: against 64 bits at both
    ends and in the middle."""
    g = torch.Generator("cuda").manual_seed(bits)
    flat = lambda scale: torch.randn(n, generator=g, device="cuda") * scale
    p, grad, m = flat(1.0), flat(1e-3), flat(1e-3)
    if bits == 32:
        s = fq.AdamWStates([p], 32, None, [m], [(m * 3).square() + 1e-9])
    else:
        (q, d), (r, e) = (fq.fp8_block_quant_rowwise(v.to(BF16)[None]) for v in (m, m.abs() * 3 + 1e-4))
        s = fq.AdamWStates([p], 8, None, [q[0].contiguous()], [r[0].contiguous()], [d[:, 0].contiguous()], [e[:, 0].contiguous()])
    cuts = [(0, 5000), (n // 256 * 128, n // 256 * 128 + 5000), (n // 128 * 128 - 4992, n)]
    part = lambda t, a, b: t[a:b].cpu().double()
    blocks = lambda t, a, b: t[a // 128:-(-b // 128)].cpu()
    before = [(part(p, a, b),) + ((part(s.exp_avg[0], a, b), part(s.exp_avg_sq[0], a, b)) if bits == 32 else
              (al.decode(s.exp_avg[0][a:b], blocks(s.exp_avg_scales[0], a, b)),
               al.decode(s.exp_avg_sq[0][a:b], blocks(s.exp_avg_sq_scales[0], a, b)).square())) for a, b in cuts]
    fq.adamw_step(s, [grad], 7, 1e-2)
    words = al.words(7, 0, n)
    for (a, b), (p0, m0, v0) in zip(cuts, before):
        p1, off_p, m1, off_m, v1, off_v = al.step64(p0, part(grad, a, b), m0, v0, 7, 1e-2, (0.9, 0.999), 1e-8, 0.01)
        assert bool(((part(p, a, b) - p1).abs() <= off_p).all())
        if bits == 32:
            assert bool(((part(s.exp_avg[0], a, b) - m1).abs() <= off_m).all())
            assert bool(((part(s.exp_avg_sq[0], a, b) - v1).abs() <= off_v).all())
            continue
        b -= (b - a) % 128 if b < n else 0  # whole blocks
        k, r = b - a, torch.sqrt(v1)
        off_r = torch.maximum(torch.sqrt(v1 + off_v) - r, r - torch.sqrt((v1 - off_v).clamp(min=0))) + 2 * al.U * r
        al.check_kept(s.exp_avg[0][a:b], blocks(s.exp_avg_scales[0], a, b), m1[:k], off_m[:k], words[a:b], False)
        al.check_kept(s.exp_avg_sq[0][a:b], blocks(s.exp_avg_sq_scales[0], a, b), r[:k], off_r[:k], words[a:b], True)


def test_a_step_is_seen_by_what_torch_has_recorded(fq):
    """A parameter that was saved for a backward pass and then stepped is a parameter that was changed."""
    p = torch.nn.Parameter(normal(100, 1))
    loss = (p * p).sum()
    s = fq.AdamWStates([p], 32)
    fq.adamw_step(s, [torch.ones(100, device="cuda")], 1, 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
