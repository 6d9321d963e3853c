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
@pytest.mark.parametrize("groups,kept,topn", [(1, 1, 1), (4, 2, 2)])
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


@pytest.mark.parametrize("score,renormalize", KINDS)
def test_one_short_group(score, renormalize):
    logits = torch.tensor([[1, .5, .2, .1, 3, 2, -INF, -INF], [3, -INF, NAN, 2, 1, 1, 1, 1], [0, 0, 0, 0, -INF, -INF, -INF, -INF],
                           [-INF] * 8, [-INF, 1, -INF, -INF, -INF, -INF, -INF, -INF]])
    _check(logits, None, 4, score, renormalize, groups=2, kept=1, topn=1)
    _check(logits, torch.linspace(0.1, -0.1, 8), 4, score, renormalize, groups=2, kept=1, topn=2, scale=2.5)


@pytest.mark.parametrize("score,renormalize", KINDS)
@pytest.mark.parametrize("E,groups,kept,k", [(64, 8, 1, 5), (93, 3, 1, 8), (160, 32, 2, 6), (128, 4, 1, 16), (256, 8, 4, 8), (256, 2, 1, 16)])
def test_short_groups(E, groups, kept, k, score, renormalize):
    """Rows whose kept groups hold fewer unmasked experts than slots, while dropped groups hold others."""
    T, per = 37, E // groups
    g = torch.Generator().manual_seed(E + k)
    logits = torch.randn(T, E, generator=g) - 4.0
    for t in range(T):
        strong = torch.randperm(groups, generator=g)[:kept]
        for i, q in enumerate(strong.tolist()):
            row = logits[t, q * per:(q + 1) * per]
            row[:] = NAN if t % 3 == 1 else -INF
            if i == 0 or t % 2:
                row[int(torch.randint(per, (1,), generator=g))] = 3.0 + float(torch.rand(1, generator=g))
        if t % 5 == 0:                     # some masked experts outside, too
            logits[t, torch.randperm(E, generator=g)[:E // 8]] = -INF
    ids, real = _chosen(logits, None, k, score, groups, kept, 1)
    lowest = torch.isfinite(logits).int().argmax(1)
    assert int(((real < k) & (lowest < ids.gather(1, real.clamp(max=k - 1)[:, None]).squeeze(1))).sum()) > 5
    _check(logits, None, k, score, renormalize, groups, kept, 1)
    _check(logits, torch.randn(E, generator=g) * 1e-3, k, score, renormalize, groups, kept, 1, 2.5)


@pytest.mark.parametrize("score,renormalize", KINDS)
def test_balanced_route_and_its_gradient(score, renormalize):
    """The whole gate, with a logit bias that masks experts: a product, the choice, and the gradient of the weights."""
    B = _B()
    T, H, E, k, groups = 61, 256, 64, 6, 8
    g = torch.Generator().manual_seed(9)
    x, wr = torch.randn(T, H, generator=g).to(torch.bfloat16), (torch.randn(E, H, generator=g) * H ** -0.5).to(torch.bfloat16)
    lb = torch.randn(E, generator=g) * 0.1
    lb[16:24] += 4.0
    lb[17:24] = -INF                       # the best group is left with one expert
    rp = B.route_params(E, k, score, renormalize, groups, 1, 1, 1.5)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    logits, load = torch.empty(T, E, device=DEV), torch.zeros(E, dtype=torch.int32, device=DEV)
    ws = torch.empty(max(256, B.moe_route_workspace_size(T, H, E)), dtype=torch.uint8, device=DEV)
    B.moe_route_balanced(x.to(DEV), wr.to(DEV), rp, ids, w, ws, load=load, logits_out=logits, logit_bias=lb.to(DEV))
    l, dw = logits.cpu(), torch.randn(T, k, generator=g)
    rid, rw, rload, rg, bound = _reference(l, None, k, dw, score, renormalize, groups, 1, 1, 1.5)
    assert int(((rw == 0).sum(1) == k - 1).sum()) > T // 2
    assert torch.equal(ids.cpu(), rid) and torch.equal(load.cpu(), rload)
    assert ((w.cpu().double() - rw).abs() <= 1.01 * O.U * rw + 2.0 ** -149).all()
    dl = torch.empty(T, E, device=DEV)
    B.moe_route_backward(logits, ids, dw.to(DEV), rp, dl)
    assert ((dl.cpu().double() - rg).abs() <= bound + O.rounding(torch.float32, rg)).all()


@pytest.mark.parametrize("score,renormalize", KINDS)
def test_train_layer_with_masked_experts(score, renormalize):
    """TrainLayer with groups and -inf in logit_bias against 64-bit autograd at the experts of the header's rule."""
    import workloads as W
    from combine_dual_overlap_amd import TrainLayer
    cfg = W.get_config(1, small=True).replace(k=3, n_groups=2, topk_groups=1, group_topn=1, score=score, renormalize=renormalize)
    inp = W.make_inputs(cfg, 5)
    inp["forced_ids"] = None
    lb = torch.zeros(cfg.E)
    lb[4:] = torch.tensor([3.0, 2.0, -INF, -INF])      # two experts in the second group, which most tokens prefer
    inp["logit_bias"], inp["select_bias"] = lb, torch.zeros(cfg.E)
    layer = TrainLayer(inp)
    x = inp["x"].to(DEV)
    dout = torch.randn(x.shape, generator=torch.Generator().manual_seed(8))
    out = layer.forward(x).clone()
    logits, ids = layer.buf["logits"][:cfg.T].cpu(), layer.buf["ids"][:cfg.T].cpu().long()
    rid, real = _chosen(logits, None, cfg.k, score, 2, 1, 1)
    assert int((real < cfg.k).sum()) > cfg.T // 2
    assert torch.equal(ids, rid)
    dx = layer.backward(dout.to(DEV))
    P = {n: t.cpu().double().requires_grad_(True) for n, t in layer.weights.items()}
    x64 = inp["x"].double().requires_grad_(True)
    masked = ~torch.isfinite(lb)[None].expand(cfg.T, cfg.E)
    l = x64 @ P["w_router"][0].T + torch.where(masked, torch.zeros_like(lb), lb).double()
    w = _weights(l, masked, ids, real, score, renormalize, cfg.routed_scale)
    y = torch.zeros_like(x64)
    for e in range(cfg.E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        a, b = (x64[t] @ P["w13"][e].T).chunk(2, dim=1)
        y = y.index_add(0, t, (a * torch.sigmoid(a) * b) @ P["w2"][e].T * w[t, j, None])
    grads = torch.autograd.grad((y * dout.double()).sum(), [x64, *P.values()])
    # fp32: five products of at most 256 terms one after the other, each off by at most terms * 2^-24: 8e-5
    near = lambda a, r: float((a.cpu().double() - r).norm() / r.norm()) < 8e-5
    assert near(out, y.detach()) and near(dx, grads[0])
    for n, r in zip(P, grads[1:]):
        assert near(layer.grads[n], r), n


@pytest.mark.parametrize("renormalize", [False, True])
def test_scores_below_fp32(renormalize):
    """Sigmoid scores whose weights are ordinary numbers only because they are divided by their sum."""
    g = torch.Generator().manual_seed(6)
    logits = torch.cat([torch.randn(1, 64, generator=g) + s for s in (-30.0, -60, -86, -90, -95, -100, -110, -200, -600)])
    logits = torch.cat([logits, logits + 20 * torch.rand(logits.shape, generator=g)])
    _check(logits, None, 6, "sigmoid", renormalize)
    _check(logits, None, 6, "sigmoid", renormalize, groups=8, kept=3, topn=2, scale=2.5)


@pytest.mark.parametrize("renormalize", [False, True])
def test_softmax_scores_below_fp32(renormalize):
    """A bias that keeps a token from its one large expert: the others' weights are ordinary once divided by their sum."""
    g = torch.Generator().manual_seed(7)
    logits = torch.cat([torch.randn(4, 64, generator=g) + s for s in (-10.0, -40, -60, -90, -104, -120, -600)])
    logits[:, 9] = 0.0
    bias = torch.zeros(64)
    bias[9] = -2.0
    _check(logits, bias, 6, "softmax", renormalize)
    _check(logits, bias, 6, "softmax", renormalize, groups=8, kept=3, topn=2, scale=2.5)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [8, 64, 200])
def test_balance_loss_of_scores_below_fp32(E, dt):
    """q = p / sum p is an ordinary number, however small a token's sigmoid scores are."""
    B = _B()
    g = torch.Generator().manual_seed(E)
    rows = [torch.randn(1, E, generator=g) + s for s in (-20.0, -60, -88, -90, -95, -100, -104, -110, -200, -1000)]
    rows += [r + 30 * torch.rand(1, E, generator=g) for r in rows]
    logits = torch.cat(rows)
    logits = torch.cat([logits, logits, logits])
    n = len(rows)
    logits[n:2 * n, 1:] = -INF                           # one expert each
    logits[2 * n:, ::2] = NAN
    T = logits.shape[0]
    load = torch.randint(0, 50, (E,), generator=g, dtype=torch.int32)
    load[0] += 1
    before = (torch.randn(T, E, generator=g) * 0.01 / T).to(dt)
    coef = 0.25
    d, loss = before.to(DEV), torch.full((1,), NAN, device=DEV)
    ws = torch.empty(B.moe_route_balance_loss_workspace_size(T, E), dtype=torch.uint8, device=DEV)
    B.moe_route_balance_loss(logits.to(DEV), load.to(DEV), B.route_params(E, 1, "sigmoid"), coef, loss, d, ws, accumulate=True)
    masked = ~torch.isfinite(logits)
    l = torch.where(masked, torch.zeros_like(logits), logits).double()
    q = torch.softmax(torch.nn.functional.logsigmoid(l).masked_fill(masked, -INF), 1)
    f = load.double() * (E / int(load.sum()))
    inner = (q * f).sum(1, keepdim=True)
    want = before.double() + coef / T * q * (f - inner) * torch.sigmoid(-l)
    # q: the argument of its exponential is off by half a step for each unit that it is long, and a few more of the
    # exponentials, the sum (pairs) and the division; f - 1 and the inner sum carry such an error of their own
    top = l.masked_fill(masked, -INF).amax(1, keepdim=True)
    far = torch.where(masked, torch.zeros_like(l), (top - l + l.abs()).clamp(max=208.0))
    err = 48 + 2 * far
    bound = coef / T * O.U * q * (err * ((f - 1).abs() + (inner - 1).abs()) + ((q * err) * (f - 1).abs()).sum(1, keepdim=True))
    assert ((d.cpu().double() - want).abs() <= bound + O.U * want.abs() + O.rounding(dt, want) + 1e-45).all()
    assert abs(loss.item() - coef / T * float((q * f).sum())) <= 4 * O.U * coef / T * float((q * (f - 1).abs() * err).sum() + T)
