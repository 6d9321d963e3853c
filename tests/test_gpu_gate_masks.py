"""Rows of the balanced gate that leave experts out, and scores at fp32's lower end: what is chosen, the gradient of its
weights, and the balance loss, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import block_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = math.inf, math.nan


def _B():
    from combine_dual_overlap_amd import binding
    return binding


def _chosen(logits, bias, k, score, groups, kept, topn):
    """(ids, real): a token's experts by the header's rule, and how many slots found a candidate.  Where candidates run
    out the masked experts follow, lowest index first."""
    T, E = logits.shape
    p, masked = O.scores(logits, score)
    key = p + (0.0 if bias is None else bias.double().numpy())
    per = E // groups
    ids, real = np.zeros((T, k), np.int64), np.zeros(T, np.int64)
    for t in range(T):
        best = np.full(groups, -np.inf)
        for g in range(groups):
            mine = np.sort(key[t, g * per:(g + 1) * per][~masked[t, g * per:(g + 1) * per]])[::-1][:topn]
            if mine.size:
                best[g] = sum(mine[1:], mine[0])
        keep = np.argsort(-best, kind="stable")[:kept]
        cand = [e for e in range(E) if not masked[t, e] and (groups == 1 or e // per in keep)]
        order = sorted(cand, key=lambda e: (-key[t, e], e))[:k]
        real[t] = len(order)
        ids[t] = order + np.flatnonzero(masked[t])[:k - len(order)].tolist()
    return torch.from_numpy(ids), torch.from_numpy(real)


def _weights(l, masked, ids, real, score, renormalize, scale):
    """Weights in 64 bits, differentiable in l (the logits, 0 where masked); slots from `real` on are the constant 0."""
    if score == "sigmoid":
        logp = torch.nn.functional.logsigmoid(l)
    else:
        logp = torch.log_softmax(l.masked_fill(masked, -1e300), 1)
    logp = logp.gather(1, ids)
    there = torch.arange(ids.shape[1])[None] < real[:, None]
    logp = torch.where(there, logp, torch.full_like(logp, -INF))
    if renormalize:
        top = logp.detach().amax(1, keepdim=True)
        e = torch.exp(logp - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
        w = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = torch.exp(logp)
    return torch.where(there, w, torch.zeros_like(w)) * scale


def _reference(logits, bias, k, dw, score, renormalize, groups, kept, topn, scale):
    """ids, weights, load, dlogits and a bound on what fp32 adds to these."""
    T, E = logits.shape
    masked = torch.from_numpy(O.scores(logits, score)[1])
    ids, real = _chosen(logits, bias, k, score, groups, kept, topn)
    l = torch.where(masked, torch.zeros_like(logits), logits.clamp(max=torch.finfo(torch.float32).max)).double()
    l = l.nan_to_num(0.0).requires_grad_(True)
    w = _weights(l, masked, ids, real, score, renormalize, scale)
    grad, = torch.autograd.grad((w * dw.double()).sum(), l)
    there = torch.arange(k)[None] < real[:, None]
    load = torch.bincount(ids[there], minlength=E).int()
    # An entry is a sum over its slots of w (d - D) and, where the scores are not normalised again, of p D, with D the row's
    # sum of w d.  A score carries the roundings of its exponent's argument (as many half steps as the argument is long), and
    # a few more of the exponential, of sums of at most 256 terms (joined in pairs) and of two divisions.
    with torch.no_grad():
        m = w / scale
        d = (dw.double() * scale).abs()
        D = (m * d).sum(1, keepdim=True)
        mag = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, ids, m * (d + D))
        p = torch.from_numpy(O.scores(logits, score)[0])
        if score == "softmax":
            mag = mag + p * D
        lo = torch.where(masked, l.amax(1, keepdim=True), l)
        far = (lo.amax(1, keepdim=True) - lo).clamp(max=104.0)
        if score == "sigmoid":
            far = torch.maximum(far, lo.abs().clamp(max=104.0))
        err = (64 + 2 * far) + 2 * (m * far.gather(1, ids)).sum(1, keepdim=True)
        bound = O.U * err * mag + 2.0 ** -125 * (1 + d.sum(1, keepdim=True))
    return ids.int(), w.detach(), load, grad, bound


def _check(logits, bias, k, score, renormalize=False, groups=1, kept=1, topn=1, scale=1.0):
    B = _B()
    T, E = logits.shape
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(3))
    rid, rw, rload, rg, bound = _reference(logits, bias, k, dw, score, renormalize, groups, kept, topn, scale)
    rp = B.route_params(E, k, score, renormalize, groups, kept, topn, scale)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    load, l = torch.zeros(E, dtype=torch.int32, device=DEV), logits.to(DEV)
    B.moe_route_select(l, rp, ids, w, select_bias=None if bias is None else bias.to(DEV), load=load)
    assert torch.equal(ids.cpu(), rid)
    assert torch.equal(load.cpu(), rload)
    # held in 64 bits and rounded once; the last term: a subnormal's step
    assert ((w.cpu().double() - rw).abs() <= 1.01 * O.U * rw + 2.0 ** -149).all()
    for dt in (torch.float32, torch.bfloat16):
        dl = torch.full((T, E), NAN, dtype=dt, device=DEV)
        B.moe_route_backward(l, ids, dw.to(DEV), rp, dl)
        assert ((dl.cpu().double() - rg).abs() <= bound + O.rounding(dt, rg)).all(), dt


KINDS = [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)]


@pytest.mark.parametrize("score,renormalize", KINDS)
@pytest.mark.parametrize("groups,kept,topn", [(1, 1, 1)])
def test_rows_that_are_not_finite(score, renormalize, groups, kept, topn):
    low = torch.finfo(torch.float32).min
    logits = torch.randn(12, 80, generator=torch.Generator().manual_seed(5))
    logits[0] = -INF
    logits[1] = NAN
    logits[2, 3:] = -INF
    logits[3, 4:] = NAN
    logits[4, ::2] = NAN
    logits[5, 7] = INF
    logits[6, [5, 70]] = INF
    logits[7, 20:60] = NAN
    logits[8, 1:] = low
    logits[9, :79] = -INF
    logits[10, [1, 2, 3]] = torch.tensor([INF, NAN, -INF])
    _check(logits, None, 5, score, renormalize, groups, kept, topn)
