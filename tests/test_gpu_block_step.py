"""The example's block: norm, layer, balance loss, their gradients and the AdamW step together, against the
same block in float32 with the bf16 weights; and its paths without gradients."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from examples import block_moe_layer as m
    return m


def operands(T, H, E, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return (r(T, H).to(torch.bfloat16).cuda(), (3 * r(T, H)).to(torch.bfloat16).cuda(), (1 + 0.2 * r(H)).cuda(),
            r(T, H).cuda(), r(T, H).cuda())


@pytest.mark.parametrize("T,H,I,E,top,ends", [(96, 256, 160, 4, 2, None), (60, 400, 128, 7, 3, [11, 11, 57]), (1, 256, 128, 4, 2, None)])
def test_gradients_against_float32(ex, T, H, I, E, top, ends):
    x, residual, gain, dy, dh = operands(T, H, E, T)
    block = ex.Block(gain, ex.make(E, H, I, top, seed=T))
    seq = None if ends is None else torch.tensor(ends, dtype=torch.int32, device="cuda")
    dloss = torch.linspace(0.5, 1.0, 1 if ends is None else len(ends)).cuda() * T
    y, h, loss = block.forward(x, residual, seq)
    dx, grads = block.backward(dy, dh, dloss)

    ids = block.layer.routed[1].long()
    counts = block.balance["counts"].float()
    # the stream is one rounded sum, whose gradient is that of each of its parts
    stream = (x.float() + residual.float()).to(torch.bfloat16).float().requires_grad_()
    assert torch.equal(h.float(), stream.detach())
    leaf = lambda t: t.float().clone().requires_grad_()
    gain_r, router, w13, w2 = leaf(gain), leaf(block.layer.router), leaf(block.layer.w13.w), leaf(block.layer.w2.w)
    rows = stream * torch.rsqrt(stream.square().mean(1, keepdim=True) + EPS) * gain_r
    rows = rows + (block.normed.y.float() - rows).detach()  # the rows that were routed
    p = torch.softmax(rows @ router.t(), 1)
    w = torch.gather(p, 1, ids)
    w = w / w.sum(1, keepdim=True)
    want = torch.zeros(T, H, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gate, up = (rows[t] @ w13[e].t()).chunk(2, 1)
        want = want.index_add(0, t, ((torch.nn.functional.silu(gate) * up) @ w2[e].t()) * w[t, j][:, None])
    bounds = [0] + ([T] if ends is None else ends)
    losses = torch.stack([(counts[s] * p[a:b].sum(0)).sum() * (E / (top * max(1, b - a) ** 2)) for s, (a, b) in enumerate(zip(bounds, bounds[1:]))])
    ((want * dy).sum() + (stream * dh).sum() + (losses * dloss).sum()).backward()

    off = lambda a, b: float((a.float() - b).norm() / b.norm())
    # A result depends on at most three products one after the other, of two operands each that are rounded by
    # 2^-5.3 in the mean square: sqrt(6) 2^-5.3 = 2^-4.0.  That is a mean: over n independent numbers the ratio
    # of two norms spreads by sqrt(1 / 2n + 1 / 2n) of itself, and has to lie within four of these.  A token
    # brings as many as the least that stands between two products, and to the router's gradient, a linear
    # map of the numbers dy . o, one for each choice.
    # The gain's gradient is of products of two normals, whose squares have a variance of 9 - 1 instead of 3 - 1
    # over their mean's square: each norm spreads by sqrt(8 / n) / 2, and both share a factor: 2 / sqrt(n) at most.
    limit = lambda n, spread=1: max(2.0 ** -3.9, 2.0 ** -4.0 * (1 + 4 * spread / n ** 0.5))
    n = T * min(H, top * I)
    assert off(y, want.detach()) < limit(n)
    assert off(loss, losses.detach()) < 1e-5
    limits = limit(n), limit(n, 2), limit(T * top), limit(n), limit(n)
    for got, ref, far in zip([dx] + grads, [stream.grad, gain_r.grad, router.grad, w13.grad, w2.grad], limits):
        assert got.shape == ref.shape and off(got, ref) < far


def test_update_moves_the_weights_and_their_bytes(ex):
    T, H, I, E, top = 64, 256, 128, 4, 2
    x, residual, gain, dy, dh = operands(T, H, E, 3)
    for bits in (8, 32):
        block = ex.Block(gain.clone(), ex.make(E, H, I, top), bits)
        for _ in range(2):
            before = [p.clone() for p in block.states.params]
            block.forward(x, residual)
            _, grads = block.backward(dy, dh, torch.ones(1, device="cuda"))
            block.update(grads, 1e-3)
            for p, q in zip(block.states.params, before):
                assert not torch.equal(p, q) and bool(torch.isfinite(p).all())
            q, q_t, s = ex.fq.fp8_block_quant_weights(block.layer.w13.w.view(-1, H), E)
            assert torch.equal(block.layer.w13.forward_bytes.reshape(-1, H), q) and torch.equal(block.layer.w13.scales, s)


def test_prompt_and_decoding_against_the_training_forward(ex):
    """The prompt's products read the norm's own 8-bit rows, the training step's those of its bf16 rows; the
    few-token layer quantizes neither."""
    T, H, I, E, top = 100, 512, 256, 8, 2
    x, residual, gain, _, _ = operands(T, H, E, 5)
    block = ex.Block(gain, ex.make(E, H, I, top))
    y, h, _ = block.forward(x, residual)
    p, hp = block.prompt(x, residual)
    d, hd = block.decode(x, residual)
    assert torch.equal(h, hp) and torch.equal(h, hd)
    off = lambda a: float((a.float() - y).norm() / y.norm())
    assert off(p) < 2.0 ** -4.4 and off(d) < 2.0 ** -3.9


def test_example_runs(ex, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["block_moe_layer.py", "--tokens", "256", "--hidden", "256", "--inner", "128", "--experts", "4", "--top", "2"])
    ex.main()
    assert "training step with update" in capsys.readouterr().out


# ------------------------------------------------------------ streams, capture and replay of the calls

def test_calls_on_another_stream_and_captured(ex):
    """Norm, routing, balance loss and both gradients, captured once and replayed on new inputs, the caller's
    work between the replays; every replay against the eager calls."""
    fq = ex.fq
    T, H, E, top = 700, 1024, 16, 4
    x, residual, gain, dy, _ = operands(T, H, E, 9)
    router = (torch.randn(E, H, generator=torch.Generator().manual_seed(1)) * H ** -0.5).to(torch.bfloat16).cuda()
    dweights, dloss = torch.randn(T, top, generator=torch.Generator().manual_seed(2)).cuda(), torch.ones(2, device="cuda")
    seq = torch.tensor([300, 650], dtype=torch.int32, device="cuda")

    def run():
        n = fq.fp8_rms_norm(x, gain, residual=residual, bf16=True)
        logits = torch.empty(T, E, device="cuda")
        ids, w = fq.moe_route(n.y, router, top, logits=logits)
        loss, counts = fq.moe_balance(logits, ids, sequences=seq)
        dl = fq.moe_route_backward(logits, ids, dweights, dloss=dloss, counts=counts, sequences=seq)
        dx, dgain = fq.fp8_rms_norm_backward(dy, n.h, n.rstd, gain)
        return [n.h, n.y, n.q, n.scales, n.rstd, ids, w, loss, counts, dl, dx, dgain]

    eager = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(eager, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        g = torch.Generator("cuda").manual_seed(i)
        x.copy_(torch.randn(T, H, generator=g, device="cuda"))
        dweights.normal_(generator=g)
        seq.copy_(torch.tensor([100 * i, 650 - i], device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, run()):
            assert torch.equal(a, b), i
