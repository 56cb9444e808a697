"""The balance loss and a router's gradients in 64 bits, with bounds for 32-bit arithmetic.  Scores are
held by their logarithms, so that no sum of them leaves the range.  Test infrastructure only."""
from __future__ import annotations

import torch

U = 2.0 ** -24
TINY = 1e-37  # what vanishes below 32 bits' normal range


def log_scores(l, scoring):
    l = l.cpu().double()
    return torch.nn.functional.logsigmoid(l) if scoring == "sigmoid" else l - torch.logsumexp(l, 1, keepdim=True).nan_to_num(neginf=0)


def softmax(v):
    """Zeros for a row without a value over minus infinity."""
    m = v.amax(1, keepdim=True)
    e = torch.exp(v - torch.where(m == -torch.inf, 0.0, m))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def spans(T, sequences):
    ends = [T] if sequences is None else sequences.tolist()
    return list(zip([0] + ends[:-1], ends))


def counts_of(ids, E, T, sequences):
    ids = ids.cpu().long()
    return torch.stack([torch.bincount(v[(v >= 0) & (v < E)], minlength=E) for v in (ids[a:b].flatten() for a, b in spans(T, sequences))])


def balance(l, ids, scoring, sequences):
    """(loss [S], counts [S, E]) as a function of l that autograd can follow."""
    T, E = l.shape
    p = softmax(log_scores(l, scoring)) if not l.requires_grad else torch.softmax(
        torch.nn.functional.logsigmoid(l) if scoring == "sigmoid" else l, 1)
    counts = counts_of(ids, E, T, sequences)
    loss = torch.stack([(counts[s].double() * p[a:b].sum(0)).sum() * (E / (ids.shape[1] * (b - a) ** 2)) if b > a else p.sum() * 0
                        for s, (a, b) in enumerate(spans(T, sequences))])
    return loss, counts


def weights(l, ids, scoring, renormalize, scale):
    """moe_route's weights of valid ids, as a function of l that autograd can follow."""
    s = torch.sigmoid(l) if scoring == "sigmoid" else torch.softmax(l, 1)
    w = torch.gather(s, 1, ids.cpu().long())
    return scale * (w / w.sum(1, keepdim=True) if renormalize else w)


def errors(l, scoring):
    """(p, rel error of p, score, rel of score, slope, rel of slope) of 32-bit arithmetic: an exponential of a
    difference d is off by its argument's rounding, |d| U, and a few units."""
    l = l.cpu().double()
    v = log_scores(l, scoring)
    p = softmax(v)
    finite = lambda d: torch.where(torch.isfinite(d), d, 0.0)
    if scoring == "sigmoid":
        s, slope = torch.exp(v), torch.sigmoid(-l)
        each = U * (finite(l).abs().clamp(max=200) + 8)
    else:
        s, slope = p, torch.ones_like(p)
        each = U * (finite(l - l.amax(1, keepdim=True)).abs().clamp(max=200) + 8)
    rel = each + (p * each).sum(1, keepdim=True) + U * 40  # of the sum and its additions, quotient and product
    return p, rel, s, each if scoring == "sigmoid" else rel, slope, each if scoring == "sigmoid" else 0 * each


def additions(n):
    """Additions that a sequence's sum goes through one after the other, at most: a thread's rows, a block's, the chunks."""
    return min(n, n // 256 + 600)


def check_balance(loss, counts, l, ids, scoring, sequences):
    T, E = l.shape
    want, want_counts = balance(l.cpu().double(), ids, scoring, sequences)
    assert torch.equal(counts.cpu().long(), want_counts)
    p, rel, *_ = errors(l, scoring)
    for s, (a, b) in enumerate(spans(T, sequences)):
        if b <= a:
            assert float(loss[s]) == 0
            continue
        f = want_counts[s].double() * (E / (ids.shape[1] * (b - a) ** 2))
        bound = (f * (p * rel)[a:b].sum(0)).sum() + U * (additions(b - a) + E + 16) * want[s] + TINY
        assert abs(float(loss[s]) - float(want[s])) <= float(bound), (s, float(loss[s]), float(want[s]), float(bound))


def gradient(l, ids, dweights, scoring, renormalize, scale, dloss, counts, sequences):
    """(dlogits in 64 bits, how far 32-bit arithmetic may be from it)."""
    T, E = l.shape
    k = ids.shape[1]
    p, rel_p, s, rel_s, slope, rel_slope = errors(l, scoring)
    want, bound = torch.zeros(2, T, E, dtype=torch.float64).unbind(0)
    if dloss is not None:
        for i, (a, b) in enumerate(spans(T, sequences)):
            if b <= a:
                continue
            dp = float(dloss[i]) * E / (k * (b - a) ** 2) * counts[i].cpu().double()
            q, rq = p[a:b], rel_p[a:b]
            dot = (q * dp).sum(1, keepdim=True)
            off = (q * dp.abs() * (rq + 32 * U)).sum(1, keepdim=True)
            want[a:b] += q * slope[a:b] * (dp - dot)
            bound[a:b] += q * slope[a:b] * ((rq + rel_slope[a:b] + 5 * U) * (dp - dot).abs() + 7 * U * dp.abs() + off)
    if dweights is not None:
        ids, dw = ids.cpu().long(), dweights.cpu().double()
        times, g = torch.zeros(2, T, E + 1, dtype=torch.float64).unbind(0)
        at = torch.where((ids >= 0) & (ids < E), ids, E)
        times = times.scatter_add(1, at, torch.ones_like(dw))[:, :E]
        size = g.scatter_add(1, at, dw.abs())[:, :E]
        g = g.scatter_add(1, at, dw)[:, :E]
        size = size + 32 * U * size  # of adding up to 32 of them
        if renormalize:
            v = torch.where(times > 0, log_scores(l, scoring) + torch.log(times.clamp(min=1)), -torch.inf)
            r = softmax(v) / times.clamp(min=1)  # of one choice
            rel_r = rel_s + (r * times * rel_s).sum(1, keepdim=True) + 60 * U
            lift = U * torch.where(times > 0, torch.where(torch.isfinite(l.cpu().double()), l.cpu().double(), 0.0), 0.0).abs().amax(1, keepdim=True).clamp(max=400)
            rel_r = rel_r + 2 * lift  # where the chosen logits' own maximum is subtracted
            dot = (r * g).sum(1, keepdim=True)
            off = (r * size * (rel_r + 40 * U)).sum(1, keepdim=True)
            want += scale * slope * r * (g - times * dot)
            bound += abs(scale) * slope * r * ((rel_r + rel_slope + 6 * U) * (g - times * dot).abs() + 34 * U * size + times * (off + 2 * U * dot.abs()))
        elif scoring == "sigmoid":
            want += scale * s * slope * g
            bound += abs(scale) * s * slope * ((rel_s + rel_slope + 5 * U) * g.abs() + 34 * U * size)
        else:
            dot = (p * g).sum(1, keepdim=True)
            off = (p * size * (rel_p + 40 * U)).sum(1, keepdim=True)
            want += scale * p * (g - dot)
            bound += abs(scale) * p * ((rel_p + 6 * U) * (g - dot).abs() + 34 * U * size + off)
    return want, bound + 4 * U * want.abs()


def check_gradient(dlogits, l, *args):
    want, bound = gradient(l, *args)
    half = torch.finfo(dlogits.dtype).eps / 2
    off = (dlogits.cpu().double() - want).abs()
    size = float(want.abs().max()) if want.numel() else 0.0
    assert bool((off <= (1 + half) * bound + half * want.abs() + TINY * max(1.0, size)).all()), float((off - bound - half * want.abs()).max())
