"""Cases of the operators around the experts: routing with a selection bias
that balances the experts, the balance loss with its gradient, products of
8-bit integers grouped by expert with scales for each token and channel, and
the norms before and after the layer with its gate and residual, with their
gradients.

`run` computes them in elementary torch operations (own = False) or through
the library's entry points (own = True); `exact` gives the results in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def _binding():
    from combine_dual_overlap_amd import binding
    return binding


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # the gate of a decode step of the V2-Lite-shaped layer
        dict(name="route_select_decode", op="route_select", T=256, E=64, k=6, score="softmax", renormalize=False,
             groups=1, kept=1, topn=1, scale=1.0),
        # the R1-shaped gate: sigmoid scores, four of eight groups
        dict(name="route_select_r1", op="route_select", T=4096, E=256, k=8, score="sigmoid", renormalize=True,
             groups=8, kept=4, topn=2, scale=2.5),
        # the skewed layer's balance loss, added to the gate's gradient
        dict(name="balance_loss_skewed", op="balance_loss", T=6001, E=64, k=6, score="softmax", skew=1.2, out="bf16",
             accumulate=True),
        # the R1-shaped gate's, by itself
        dict(name="balance_loss_r1", op="balance_loss", T=4096, E=256, k=8, score="sigmoid", skew=0.3, out="f32",
             accumulate=False),
        # the down projection of a decode step of the V2-Lite-shaped layer: about 24 rows an expert
        dict(name="gemm_int8_decode", op="gemm_int8", rows=1536, experts=64, N=2048, K=1408, skew=0.0, spare=0,
             out="bf16"),
        # a dense product of the R1-shaped share's widths: one group
        dict(name="gemm_int8_dense", op="gemm_int8", rows=4096, experts=0, N=7168, K=2048, skew=0.0, spare=0,
             out="f32"),
        # the experts of a decode step, from bf16 rows
        dict(name="ffn_int8_decode", op="ffn_int8", rows=1536, experts=64, H=2048, I=1408, skew=0.0, spare=0),
        # the experts of the Qwen3-shaped prefill layer, from bf16 rows
        dict(name="ffn_int8_prefill", op="ffn_int8", rows=65536, experts=128, H=2048, I=768, skew=0.0, spare=0),
        # a decode step's way out of the layer: combine, norm, gate, residual, and the next layer's norm
        dict(name="block_out_decode", op="block_out", T=256, H=2048, k=6, local=1.0, post=True, gate="channel",
             next=True, dt="bf16"),
        # the same of the Qwen3-shaped prefill layer
        dict(name="block_out_prefill", op="block_out", T=8192, H=2048, k=8, local=1.0, post=True, gate="channel",
             next=True, dt="bf16"),
        # gradients of the norm after the Qwen3-shaped layer
        dict(name="block_backward_post", op="block_backward", kind="post", T=8192, H=2048, post=True, gate="channel",
             residual=False, dt="bf16"),
        # gradients of the norm before the R1-shaped layer, an odd number of tokens
        dict(name="block_backward_pre", op="block_backward", kind="pre", T=2047, H=7168, post=True, gate="none",
             residual=True, dt="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route_select", "route_select", "balance_loss", "gemm_int8", "gemm_int8", "ffn_int8", "block_out",
                     "block_out", "block_backward", "block_backward"])
    if op == "route_select":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = rng.randint(1 if groups == 1 else 2, 256 // groups)
        E = groups * per
        kept = rng.randint(1, groups)
        return dict(op=op, T=_log_int(rng, 1, 8192), E=E, k=rng.randint(1, min(kept * per, 16)),
                    score=rng.choice(["softmax", "sigmoid"]), renormalize=rng.random() < 0.5, groups=groups, kept=kept,
                    topn=rng.randint(1, min(per, 4)), scale=rng.choice([1.0, 2.5]))
    if op == "balance_loss":
        E = rng.randint(2, 256)
        return dict(op=op, T=_log_int(rng, 1, 8192), E=E, k=rng.randint(1, min(E, 16)),
                    score=rng.choice(["softmax", "sigmoid"]), skew=rng.choice([0.3, 0.6, 1.2]),
                    out=rng.choice(["bf16", "f32"]), accumulate=rng.random() < 0.5)
    if op in ("gemm_int8", "ffn_int8"):
        case = dict(op=op, rows=_log_int(rng, 1, 16384), experts=rng.choice([0, 1, 3, 8, 37, 64]),
                    skew=rng.choice([0.0, 0.6, 1.2]), spare=rng.choice([0, 0, 1, 70]))
        one, two = 16 * _log_int(rng, 1, 1408 // 16), 16 * _log_int(rng, 1, 2048 // 16)
        if op == "ffn_int8":
            return dict(case, H=two, I=one)
        return dict(case, N=8 * _log_int(rng, 1, 2816 // 8), K=two, out=rng.choice(["bf16", "f32"]))
    dt = rng.choice(["bf16", "bf16", "f32"])
    step = 4 if dt == "f32" else 8
    case = dict(op=op, T=_log_int(rng, 1, 4096), H=step * _log_int(rng, 1, 7168 // step), dt=dt,
                post=rng.random() < 0.8, gate=rng.choice(["none", "channel", "token", "full"]))
    if op == "block_out":
        return dict(case, k=rng.choice([0, 0, 1, 2, 6, 8]), local=rng.choice([1.0, 1.0, 0.5]), next=rng.random() < 0.6)
    if rng.random() < 0.5:
        return dict(case, kind="pre", post=True, gate="none", residual=rng.random() < 0.7)
    return dict(case, kind="post", residual=False)


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _counts(case, seed):
    """Rows of each expert: independent draws from a Zipf-like popularity (skew 0: uniform)."""
    E, rows = case["experts"], case["rows"]
    if E == 0:
        return [rows]
    g = torch.Generator().manual_seed(seed * 7 + 1)
    p = torch.arange(1, E + 1, dtype=torch.float64).pow(-case["skew"])[torch.randperm(E, generator=g)]
    return torch.bincount(torch.multinomial(p, rows, replacement=True, generator=g), minlength=E).tolist()


def _weights(normal, *shape):
    """Weights in 8 bits with a scale for each output channel."""
    w = normal(*shape, std=shape[-1] ** -0.5)
    s = w.abs().amax(-1) / 127.0
    return w.div_(s[..., None]).round_().to(torch.int8), s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]

    def normal(*shape, std=1.0, dt=torch.float32):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dt)

    s = dict(case)
    if op == "route_select":
        T, E, k = case["T"], case["E"], case["k"]
        # a popularity that the bias has begun to even out
        s.update(logits=normal(T, E) + 0.5 * normal(E), bias=normal(E, std=0.05 if case["score"] == "sigmoid" else 0.2 / E),
                 ids=torch.zeros(T, k, dtype=torch.int32, device=DEV), w=torch.zeros(T, k, device=DEV),
                 load=torch.zeros(E, dtype=torch.int32, device=DEV))
        return s
    if op == "balance_loss":
        T, E, k = case["T"], case["E"], case["k"]
        logits = normal(T, E) - case["skew"] * torch.log(torch.arange(1, E + 1, device=DEV).float())
        ids = torch.topk(logits, k, dim=1).indices
        s.update(logits=logits, load=torch.bincount(ids.flatten(), minlength=E).to(torch.int32), coef=0.01,
                 loss=torch.zeros(1, device=DEV), dlogits=normal(T, E, std=0.01 / T, dt=DT[case["out"]]))
        return s
    if op in ("gemm_int8", "ffn_int8"):
        cnt = _counts(case, seed)
        dense = case["experts"] == 0
        E, cap = len(cnt), case["rows"] + (0 if dense else case["spare"])
        s.update(counts=cnt, offsets=None if dense else
                 torch.tensor([sum(cnt[:e]) for e in range(E + 1)], dtype=torch.int32, device=DEV))
        if op == "gemm_int8":
            N, K = case["N"], case["K"]
            s["b"], s["b_scale"] = _weights(normal, E, N, K)
            s["a"], s["a_scale"] = _weights(normal, cap, K)
            s["c"] = torch.zeros(cap, N, dtype=DT[case["out"]], device=DEV)
            return s
        H, I = case["H"], case["I"]
        s["x"] = normal(cap, H, dt=torch.bfloat16)
        s["w13"], s["w13_scale"] = _weights(normal, E, 2 * I, H)
        s["w2"], s["w2_scale"] = _weights(normal, E, H, I)
        s["y"] = torch.zeros(cap, H, dtype=torch.bfloat16, device=DEV)
        return s
    T, H, dt = case["T"], case["H"], DT[case["dt"]]
    s["post_w"] = (1.0 + normal(H, std=0.1)).to(dt) if case["post"] else None
    gates = dict(none=lambda: None, channel=lambda: normal(H, std=0.3, dt=dt),
                 token=lambda: torch.rand(T, 1, generator=g, device=DEV), full=lambda: normal(T, H, std=0.3, dt=dt))
    s.update(gate=gates[case["gate"]](), shape=case["gate"], factor=0.5)
    if op == "block_out":
        k = case["k"]
        s.update(res=normal(T, H, dt=dt), out=torch.zeros(T, H, dtype=dt, device=DEV),
                 next_w=(1.0 + normal(H, std=0.1)).to(dt) if case["next"] else None,
                 n=torch.zeros(T, H, dtype=dt, device=DEV) if case["next"] else None)
        if k == 0:
            s["y"] = normal(T, H, dt=dt)
            return s
        local = torch.rand(T * k, generator=g, device=DEV) < case["local"]
        order = torch.randperm(T * k, generator=g, device=DEV)
        pos = torch.full((T * k,), -1, dtype=torch.int64, device=DEV)
        mine = order[local[order]]
        pos[mine] = torch.arange(mine.numel(), device=DEV)
        s.update(y_perm=normal(T * k, H, dt=dt), inv=pos.to(torch.int32), w=torch.rand(T, k, generator=g, device=DEV))
        return s
    y = normal(T, H, dt=dt)
    new = lambda *shape, t=torch.float32: torch.zeros(shape, dtype=t, device=DEV)
    dgates = dict(none=lambda: None, channel=lambda: new(H), token=lambda: new(T, 1), full=lambda: new(T, H, t=dt))
    s.update(d=normal(T, H, std=0.1, dt=dt), y=y, rstd=torch.rsqrt(y.float().square().mean(1) + EPS), dy=new(T, H, t=dt),
             dw=new(H) if case["post"] else None, dgate=dgates[case["gate"]](),
             dres=normal(T, H, std=0.1, dt=dt) if case["residual"] else None)
    return s


# --------------------------------------------------------------------------- plain forms

def _scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route_select(s):
    # in 64 bits: what is chosen hangs on which of two near scores is larger
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    p = _scores(s["logits"].double(), s["score"])
    key = p + s["bias"].double()
    if G > 1:
        best = torch.sort(key.reshape(T, G, E // G), dim=2, descending=True, stable=True).values[:, :, :s["topn"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["kept"]]
        mask = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        key = torch.where(mask.repeat_interleave(E // G, dim=1), key, -math.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if s["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    s["ids"].copy_(ids)
    s["w"].copy_(w * s["scale"])
    s["load"].add_(torch.zeros(E, dtype=torch.int32, device=DEV).scatter_add_(0, ids.flatten(), torch.ones_like(ids.flatten(), dtype=torch.int32)))


def _plain_balance_loss(s):
    T, E = s["T"], s["E"]
    f = s["load"].double() * (E / s["load"].sum().double())
    l = s["logits"].double()                      # sums over all tokens, differences of near values
    p = _scores(l, s["score"])
    q = p / p.sum(1, keepdim=True) if s["score"] == "sigmoid" else p
    s["loss"].copy_(s["coef"] * (f * q.sum(0)).sum().reshape(1) / T)
    d = (s["coef"] / T) * q * (f - (q * f).sum(1, keepdim=True))
    if s["score"] == "sigmoid":
        d = d * (1.0 - p)
    s["dlogits"].copy_(s["dlogits"].double() + d if s["accumulate"] else d)


def _quantize(x):
    """Codes and scales of rows: the integer nearest to x / scale, scale = amax / 127 in 32 bits."""
    scale = x.float().abs().amax(1) / 127.0
    q = torch.where(scale[:, None] > 0, torch.round(x.double() / scale.double()[:, None]), 0.0)
    return q.float(), scale


def _spans(s):
    """(expert, first row, row behind the last) of each expert that has rows."""
    at = 0
    for e, n in enumerate(s["counts"]):
        if n:
            yield e, at, at + n
        at += n


def _plain_int8(s):
    if s["op"] == "gemm_int8":
        for e, i, j in _spans(s):
            s["c"][i:j] = (s["a"][i:j].float() @ s["b"][e].float().t()) * s["a_scale"][i:j, None] * s["b_scale"][e]
        return s["c"]
    I = s["I"]
    xq, xs = _quantize(s["x"])
    for e, i, j in _spans(s):
        gu = (xq[i:j] @ s["w13"][e].float().t()) * xs[i:j, None] * s["w13_scale"][e]
        hq, hs = _quantize(gu[:, :I] / (1.0 + torch.exp(-gu[:, :I])) * gu[:, I:])
        s["y"][i:j] = (hq @ s["w2"][e].float().t()) * hs[:, None] * s["w2_scale"][e]
    return s["y"]


def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w.float()


def _plain_block_out(s):
    T, k = s["T"], s["k"]
    if k == 0:
        y = s["y"].float()
    else:
        inv = s["inv"].long().reshape(T, k)
        y = (s["y_perm"][inv.clamp(min=0)].float() * (s["w"] * (inv >= 0))[:, :, None]).sum(1)
    z = _norm(y, s["post_w"]) if s["post"] else y
    if s["gate"] is not None:
        z = z * s["gate"].float()
    out = s["res"].float() + s["factor"] * z
    s["out"].copy_(out)
    if s["next"]:
        s["n"].copy_(_norm(out, s["next_w"]))


def _plain_block_backward(s):
    d, y = s["d"].float(), s["y"].float()
    if s["kind"] == "post":
        d = d * s["factor"]
    yhat = y * s["rstd"][:, None] if s["post"] else y
    if s["gate"] is not None:
        dg = d * yhat * s["post_w"].float() if s["post"] else d * yhat
        s["dgate"].copy_(dg.sum(0) if s["shape"] == "channel" else dg.sum(1, keepdim=True) if s["shape"] == "token" else dg)
        d = d * s["gate"].float()
    if s["post"]:
        s["dw"].copy_((d * yhat).sum(0))
        d = d * s["post_w"].float()
        d = s["rstd"][:, None] * (d - yhat * (d * yhat).mean(1, keepdim=True))
    if s["residual"]:
        d = d + s["dres"].float()
    s["dy"].copy_(d)


def _plain(s):
    op = s["op"]
    if op in ("gemm_int8", "ffn_int8"):
        _plain_int8(s)
    else:
        dict(route_select=_plain_route_select, balance_loss=_plain_balance_loss, block_out=_plain_block_out,
             block_backward=_plain_block_backward)[op](s)
    return _out(s)


def _out(s):
    """What a pass has computed: the tensors that it wrote."""
    names = dict(route_select=("ids", "w", "load"), balance_loss=("loss", "dlogits"), gemm_int8=("c",), ffn_int8=("y",),
                 block_out=("out", "n"), block_backward=("dy", "dw", "dgate"))[s["op"]]
    return {n: s[n] for n in names if s[n] is not None}


# --------------------------------------------------------------------------- the library's calls

def _scratch(s, nbytes):
    """A workspace, which a caller keeps."""
    if "ws" not in s:
        s["ws"] = torch.empty(nbytes(), dtype=torch.uint8, device=DEV)
    return s["ws"]


def _own(s):
    B = _binding()
    op = s["op"]
    if op in ("route_select", "balance_loss") and "rp" not in s:
        s["rp"] = B.route_params(s["E"], s["k"], s["score"], s.get("renormalize", False), s.get("groups", 1),
                                 s.get("kept", 1), s.get("topn", 1), s.get("scale", 1.0))
    if op == "route_select":
        B.moe_route_select(s["logits"], s["rp"], s["ids"], s["w"], select_bias=s["bias"], load=s["load"])
    elif op == "balance_loss":
        ws = _scratch(s, lambda: B.moe_route_balance_loss_workspace_size(s["T"], s["E"]))
        B.moe_route_balance_loss(s["logits"], s["load"], s["rp"], s["coef"], s["loss"], s["dlogits"], ws,
                                 accumulate=s["accumulate"])
    elif op == "gemm_int8":
        B.moe_grouped_gemm_int8(s["a"], s["a_scale"], s["b"], s["b_scale"], s["offsets"], s["c"])
    elif op == "ffn_int8":
        cap, H = s["x"].shape
        ws = _scratch(s, lambda: B.moe_ffn_int8_workspace_size(cap, s["I"]))
        if "xq" not in s:
            s["xq"] = torch.empty(cap, H, dtype=torch.int8, device=DEV)
            s["xs"] = torch.empty(cap, device=DEV)
        B.moe_quant_int8_rows(s["x"], s["xq"], s["xs"])
        B.moe_grouped_ffn_int8(s["xq"], s["xs"], s["offsets"], s["w13"], s["w13_scale"], s["w2"], s["w2_scale"], s["y"], ws)
    elif op == "block_out":
        more = dict(post_w=s["post_w"], gate=s["gate"], scale=s["factor"], next_w=s["next_w"], next_n=s["n"])
        if s["k"] == 0:
            B.moe_post_norm(s["y"], s["res"], s["out"], EPS, **more)
        else:
            B.moe_combine_post_norm(s["y_perm"], s["inv"], s["w"], s["res"], s["out"], EPS, **more)
    else:
        ws = _scratch(s, lambda: B.moe_norm_backward_workspace_size(s["T"], s["H"]))
        if s["kind"] == "pre":
            B.moe_pre_norm_backward(s["d"], s["y"], s["rstd"], s["post_w"], s["dy"], s["dw"], ws, dres=s["dres"])
        else:
            B.moe_post_norm_backward(s["d"], s["y"], s["dy"], ws, rstd=s["rstd"] if s["post"] else None,
                                     post_w=s["post_w"], dpost_w=s["dw"], gate=s["gate"], dgate=s["dgate"],
                                     scale=s["factor"])
    return _out(s)


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------- what each case cannot do without

def work(case):
    op = case["op"]
    if op == "route_select":
        T, E, k = case["T"], case["E"], case["k"]
        return dict(bytes=T * (4 * E + 8 * k) + 12 * E, flops=T * E * 4)
    if op == "balance_loss":
        T, E = case["T"], case["E"]
        z = 4 if case["out"] == "f32" else 2
        return dict(bytes=T * E * (4 + z * (2 if case["accumulate"] else 1)) + 4 * E + 4, flops=T * E * 8)
    if op in ("gemm_int8", "ffn_int8"):
        M, E = case["rows"], max(1, case["experts"])
        used = min(E, M)                                        # experts with rows, about
        if op == "gemm_int8":
            N, K = case["N"], case["K"]
            return dict(bytes=M * K + used * N * (K + 4) + M * N * (4 if case["out"] == "f32" else 2) + 4 * M,
                        flops=2 * M * N * K)
        H, I = case["H"], case["I"]
        return dict(bytes=4 * M * H + used * (3 * I * H + 8 * I + 4 * H), flops=6 * M * H * I)
    T, H, z = case["T"], case["H"], 4 if case["dt"] == "f32" else 2
    row, full = T * H * z, case["gate"] == "full"
    if op == "block_out":
        rows = max(1, case["k"]) * (case["local"] if case["k"] else 1)
        return dict(bytes=int(row * (rows + 2 + case["next"] + full)) + 8 * T * case["k"] + 3 * H * z,
                    flops=int(T * H * (2 * rows + 8)))
    return dict(bytes=row * (3 + case["residual"] + 2 * full) + 4 * T + H * (z + 4), flops=10 * T * H)


# --------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route_select":
        T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
        l = s["logits"].double()
        p = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
        key, lowest = p + s["bias"], torch.finfo(torch.float64).min
        allowed = torch.ones(T, E, dtype=torch.bool, device=DEV)
        if G > 1:
            best = torch.topk(key.view(T, G, -1), case["topn"], dim=2).values.sum(2)
            order = (best[:, :, None] < best[:, None, :]).sum(2)       # groups that are better
            allowed = (order < case["kept"]).repeat_interleave(E // G, dim=1)
        taken = key.masked_fill(~allowed, lowest)
        ids = torch.zeros(T, k, dtype=torch.int64, device=DEV)
        for j in range(k):
            ids[:, j] = taken.argmax(1)
            taken[torch.arange(T, device=DEV), ids[:, j]] = lowest
        w = torch.gather(p, 1, ids)
        w = (w / w.sum(1, keepdim=True) if case["renormalize"] else w) * case["scale"]
        return dict(ids=ids.int(), w=w, load=torch.bincount(ids.flatten(), minlength=E).int())
    if op == "balance_loss":
        l = s["logits"].double().requires_grad_(True)
        p = torch.softmax(l, 1)
        if case["score"] == "sigmoid":
            p = torch.sigmoid(l)
            p = p / p.sum(1, keepdim=True)
        share = s["load"].double() / float(s["load"].sum())
        loss = s["coef"] * case["E"] * torch.dot(share, p.mean(0))
        d = torch.autograd.grad(loss, l)[0]
        return dict(loss=loss.detach().reshape(1), dlogits=s["dlogits"].double() + d if case["accumulate"] else d)
    if op in ("gemm_int8", "ffn_int8"):
        out = (s["c"] if op == "gemm_int8" else s["y"]).double()
        first = 0

        def product(a, a_scale, b, b_scale):
            return torch.matmul(a * a_scale.double().unsqueeze(1), (b.double() * b_scale.double().unsqueeze(1)).T.contiguous())

        def integers(x):
            unit = (x.abs().max(dim=1).values.float() / 127).double()       # a scale is held in 32 bits
            return torch.round(x / unit.clamp(min=1e-300).unsqueeze(1)), unit

        for e, n in enumerate(s["counts"]):
            r = slice(first, first + n)
            first += n
            if n == 0:
                continue
            if op == "gemm_int8":
                out[r] = product(s["a"][r].double(), s["a_scale"][r], s["b"][e], s["b_scale"][e])
                continue
            q, unit = integers(s["x"][r].double())
            gate, up = product(q, unit, s["w13"][e], s["w13_scale"][e]).chunk(2, dim=1)
            q, unit = integers(gate * torch.sigmoid(gate) * up)
            out[r] = product(q, unit, s["w2"][e], s["w2_scale"][e])
        return dict(c=out) if op == "gemm_int8" else dict(y=out)

    def normed(x, w):
        return x / torch.sqrt((x * x).sum(1, keepdim=True) / case["H"] + EPS) * w

    if op == "block_out":
        if case["k"] == 0:
            y = s["y"].double()
        else:
            y = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV)
            inv = s["inv"].view(case["T"], case["k"])
            for j in range(case["k"]):
                t = torch.nonzero(inv[:, j] >= 0).flatten()
                y[t] += s["w"][t, j, None].double() * s["y_perm"][inv[t, j].long()].double()
        if case["post"]:
            y = normed(y, s["post_w"].double())
        out = s["res"].double() + y * 0.5 * (1.0 if s["gate"] is None else s["gate"].double())
        return dict(out=out, n=normed(out, s["next_w"].double())) if case["next"] else dict(out=out)
    # the gradient of <d, factor * gate * norm(y) * w>; the factor is the layer's alone
    leaf = {n: s[n].double().requires_grad_(True) for n in ("y", "post_w", "gate") if s[n] is not None}
    z = normed(leaf["y"], leaf["post_w"]) if case["post"] else leaf["y"] * 1.0
    z = z * leaf.get("gate", 1.0) * (0.5 if case["kind"] == "post" else 1.0)
    grads = dict(zip(leaf, torch.autograd.grad(z, list(leaf.values()), s["d"].double())))
    out = dict(dy=grads["y"] + s["dres"].double() if case["residual"] else grads["y"])
    if case["post"]:
        out["dw"] = grads["post_w"]
    if s["gate"] is not None:
        out["dgate"] = grads["gate"]
    return out
