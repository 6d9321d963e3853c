"""64-bit forms of the balanced gate, the balance loss, the 8-bit integer products
and the norms around the layer, on the CPU, with bounds on what fp32 arithmetic
may add.  U is half a step of fp32 at 1."""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}      # half a step, relative


def rounding(dtype, value):
    """Largest rounding error of `value` in dtype (the last term: subnormal steps)."""
    return HALF[dtype] * value.abs() + torch.finfo(dtype).tiny * HALF[dtype]


# ------------------------------------------------------------------ gate

def scores(logits, score):
    """(p, masked) of logits [T, E]: -inf and NaN are masked, +inf is the largest finite one."""
    l = logits.double().numpy()
    masked = ~(l > -np.inf)
    l = np.where(masked, 0.0, np.minimum(l, np.finfo(np.float32).max))
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            p = 1.0 / (1.0 + np.exp(-l))
    else:
        top = np.where(masked, -np.inf, l).max(1, keepdims=True)
        with np.errstate(under="ignore"):
            e = np.where(masked, 0.0, np.exp(l - np.where(np.isfinite(top), top, 0.0)))
        s = e.sum(1, keepdims=True)
        p = np.divide(e, s, out=np.zeros_like(e), where=s > 0)
    return np.where(masked, 0.0, p), masked


def select(logits, bias, k, score, renormalize=False, groups=1, kept=1, topn=1, scale=1.0):
    """(ids, weights, load) as the header states them, one token at a time."""
    T, E = logits.shape
    p, masked = scores(logits, score)
    key = p + (0.0 if bias is None else bias.double().numpy())
    ids, w, load = np.zeros((T, k), np.int32), np.zeros((T, k)), np.zeros(E, np.int32)
    per = E // groups
    for t in range(T):
        cand = [e for e in range(E) if not masked[t, e]]
        if groups > 1:
            best = []
            for g in range(groups):
                mine = sorted((key[t, e] for e in cand if e // per == g), reverse=True)[:topn]
                best.append(sum(mine[1:], mine[0]) if mine else -np.inf)
            keep = sorted(range(groups), key=lambda g: (-best[g], g))[:kept]
            cand = [e for e in cand if e // per in keep]
        order = sorted(cand, key=lambda e: (-key[t, e], e))[:k]
        rest = [e for e in range(E) if e not in order]
        real = len(order)
        order = order + rest[:k - real]
        ids[t] = order
        w[t, :real] = p[t, order[:real]]
        load[order[:real]] += 1
        if renormalize and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return torch.from_numpy(ids), torch.from_numpy(w * scale), torch.from_numpy(load)


def balance_loss(logits, load, coef, score):
    """(loss, dlogits, bound on what fp32 adds to dlogits)."""
    T, E = logits.shape
    p, _ = scores(logits, score)
    p = torch.from_numpy(p)
    s = p.sum(1, keepdim=True)
    q = torch.where(s > 0, p / s.clamp(min=1e-300), torch.zeros_like(p))
    total = int(load.sum())
    f = load.double() * (E / total) if total else torch.zeros(E, dtype=torch.float64)
    loss = coef * float((q * f).sum()) / max(T, 1)
    inner = (q * f).sum(1, keepdim=True) / torch.where(s > 0, q.sum(1, keepdim=True), torch.ones_like(s))
    d = coef / max(T, 1) * q * (f - inner)
    if score == "sigmoid":
        d = d * (1.0 - p)
    # q: its exponent's argument is off by |l - max| half steps and the exponential, the sum and the division by a few;
    # f - 1 and the inner sum each carry such an error of their own
    l = logits.double().clamp(-80, 80).nan_to_num()
    err = 24 + 2 * (l - l.amax(1, keepdim=True)).abs() + 2 * l.abs()
    mag = (f - 1).abs() + ((q * err).sum(1, keepdim=True) * (f - 1).abs().max()) / 24
    bound = coef / max(T, 1) * q * err * U * 2 * mag + 1e-45
    return loss, d, bound


# ------------------------------------------------------------------ integers

INV127 = np.float32(1.0) / np.float32(127.0)


def quantize(x):
    """(codes, scales) of rows x [n, K] (float32 values): exact."""
    x = x.float().numpy()
    amax = np.abs(x).max(1)
    with np.errstate(invalid="ignore"):
        scale = (amax * INV127).astype(np.float32)
    bad = ~np.isfinite(x).all(1)
    scale[bad] = np.nan
    q = np.zeros(x.shape, np.float64)
    ok = ~bad & (scale > 0)
    q[ok] = np.clip(np.rint(x[ok].astype(np.float64) / scale[ok].astype(np.float64)[:, None]), -127, 127)
    return torch.from_numpy(q).to(torch.int8), torch.from_numpy(scale)


def int8_product(a, a_scale, b, b_scale):
    """The product's fp32 values, bit for bit: exact sums, then three fp32 roundings.  (Whole numbers below 2^53.)"""
    acc = (a.double() @ b.double().t()).numpy().astype(np.float32)
    return torch.from_numpy((acc * a_scale.numpy()[:, None]).astype(np.float32) * b_scale.numpy()[None, :])


def swiglu_int8(xq, xs, w13, s13):
    """(h, bound) in 64 bits of one expert."""
    g, u = (xq.double() @ w13.double().t() * xs.double()[:, None] * s13.double()).chunk(2, dim=1)
    h = g * torch.sigmoid(g) * u
    # g and u: three roundings each; silu's relative slope is at most 1 + |g|, its exponential is off by |g| log2 e + 2
    # (once e^-g passes fp32's range, below g = -88.7, the sigmoid 1 / (1 + e^-g) is 0 where it is e^g < 2^-127: h is
    # then off by |g u| 2^-127)
    return h, h.abs() * U * (16 + 8 * g.abs()) + (g * u).abs() * 2.0 ** -126 + 1e-37


def ffn_int8(xq, xs, w13, s13, w2, s2):
    """(y, bound): the codes of h that stand within its error of a half may be one off."""
    h, err = swiglu_int8(xq, xs, w13, s13)
    amax = h.abs().amax(1)
    scale = (amax.float() * float(INV127)).double()
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    v = h / scale[:, None]
    q = torch.round(v)
    near = ((v - torch.floor(v) - 0.5).abs() <= err / scale[:, None] + v.abs() * (err / h.abs().clamp(min=1e-300)).amax(1, keepdim=True) + 1e-6)
    w = w2.double()
    y = q @ w.t() * scale[:, None] * s2.double()
    flips = near.double() @ w.abs().t() * scale[:, None] * s2.double()
    rel = (err / h.abs().clamp(min=1e-300)).amax(1, keepdim=True)          # of the row's scale
    return y, flips + y.abs() * (rel + 8 * U)


# ------------------------------------------------------------------ norms

def combine(y_perm, inv, w, shared=None):
    """(y, sum of magnitudes) [T, H]."""
    T, k = w.shape
    inv = inv.long().view(T, k)
    rows = y_perm.double()[inv.clamp(min=0)] * (w.double() * (inv >= 0))[:, :, None]
    y, mag = rows.sum(1), rows.abs().sum(1)
    if shared is not None:
        y, mag = y + shared.double(), mag + shared.double().abs()
    return y, mag


C = 128 * U      # fewer than 100 roundings lie between a row and its outputs: 32 + 22 in a row's sum, the root, the factors


def norm(x, mag, w, eps):
    """(x r w, its bound, r); mag: magnitude that x's own error is C times of."""
    r = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    n = x * r * w
    # r moves by the relative error of the mean square, at most that of the largest terms: 2 C sum(mag |x|) / sum x^2
    dr = C * (1 + (mag * x.abs()).sum(1, keepdim=True) / ((x * x).sum(1, keepdim=True) + eps * x.shape[1]))
    return n, C * (mag * r * w.abs()) + dr * n.abs(), r.squeeze(1)


def block_out(y, mag, res, eps, post_w=None, gate=None, scale=1.0, next_w=None):
    """dict of out, n, rstd, next_rstd and the bounds of out and n before their rounding."""
    z, bz, r = (y, C * mag, None) if post_w is None else norm(y, mag, post_w.double(), eps)
    g = 1.0 if gate is None else gate.double()
    out = scale * g * z
    bound = abs(scale) * (torch.as_tensor(g).abs() * (bz + C * z.abs()))
    if res is not None:
        out = out + res.double()
        bound = bound + C * out.abs() + 2 * U * res.double().abs()
    d = dict(out=out, out_bound=bound, rstd=r)
    if next_w is not None:
        n, bn, r2 = norm(out, bound / C, next_w.double(), eps)
        d.update(n=n, n_bound=bn, next_rstd=r2)
    return d


def norm_backward(d, y, rstd, w, gate, kind, scale, dres):
    """dict name -> (value, bound) of the gradients of <d, scale gate (y rstd w)> plus dres, by the formula."""
    d, y = d.double() * scale, y.double()
    H = y.shape[1]
    yh = y * rstd.double()[:, None] if w is not None else y
    wd = w.double() if w is not None else torch.ones(H, dtype=torch.float64)
    g = gate.double() if gate is not None else torch.ones(1, 1, dtype=torch.float64)
    q = d * g * wd
    out = {}
    if w is not None:
        m = (q * yh).mean(1, keepdim=True)
        dy = rstd.double()[:, None] * (q - yh * m)
        bound = C * rstd.double()[:, None] * (q.abs() + yh.abs() * (q * yh).abs().mean(1, keepdim=True))
        out["dw"] = ((d * g * yh).sum(0), C * (d * g * yh).abs().sum(0))
    else:
        dy, bound = q, C * q.abs()
    if dres is not None:
        dy, bound = dy + dres.double(), bound + C * (dy.abs() + dres.double().abs())
    out["dy"] = (dy, bound)
    if gate is not None:
        dg = d * yh * wd
        if kind == "full":
            out["dgate"] = (dg, C * dg.abs())
        else:
            axis = 0 if kind == "channel" else 1
            out["dgate"] = (dg.sum(axis, keepdim=axis == 1), C * dg.abs().sum(axis, keepdim=axis == 1))
    return out
