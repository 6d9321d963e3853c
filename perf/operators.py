"""Cases of the training operators of the MoE layer: the grouped matrix
products (with their SwiGLU epilogues), the gradients of the combine and of
the router's gate, and the AdamW step.

`run` computes them in elementary torch operations (own = False) or through
the library's entry points (own = True); `exact` gives the results in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _binding():
    from combine_dual_overlap_amd import binding
    return binding


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # the gate/up product of a decode step of the V2-Lite-shaped layer: about 24 rows an expert
        dict(name="swiglu_decode", op="swiglu", rows=1536, experts=64, H=2048, I=1408, skew=0.0, spare=0, dt="bf16"),
        # the down projection of the skewed layer (Zipf popularity, one expert never chosen)
        dict(name="nt_down_skewed", op="gemm", kind="nt", rows=36006, experts=64, N=2048, K=1408, skew=1.2, spare=0,
             dt="bf16", out="bf16", accumulate=False),
        # backward through down projection and SwiGLU of the Qwen3-shaped prefill layer
        dict(name="swiglu_backward_prefill", op="swiglu_backward", rows=65536, experts=128, H=2048, I=768, skew=0.0,
             spare=0, dt="bf16"),
        # the weight gradient of the skewed layer's gate/up matrices
        dict(name="tn_gate_up_skewed", op="gemm", kind="tn", rows=36006, experts=64, N=2816, K=2048, skew=1.2, spare=0,
             dt="bf16", out="bf16", accumulate=False),
        # the router's weight gradient of the R1-shaped share: one dense group, few tiles, a long reduction
        dict(name="tn_router_dense", op="gemm", kind="tn", rows=4096, experts=0, N=256, K=7168, skew=0.0, spare=0,
             dt="bf16", out="f32", accumulate=True),
        # the tiny fp32 layer's gradient of its dispatched rows: latency
        dict(name="nn_tiny_f32", op="gemm", kind="nn", rows=128, experts=8, N=128, K=512, skew=0.0, spare=5, dt="f32",
             out="f32", accumulate=False),
        # a decode-sized step of the V2-Lite-shaped layer
        dict(name="combine_backward_decode", op="combine_backward", T=256, H=2048, k=6, local=1.0, dt="bf16"),
        # the Qwen3-shaped prefill layer
        dict(name="combine_backward_prefill", op="combine_backward", T=8192, H=2048, k=8, local=1.0, dt="bf16"),
        dict(name="route_backward_decode", op="route_backward", T=256, E=64, k=6, score="softmax", renormalize=False,
             scale=1.0, out="bf16"),
        # the R1-shaped router: sigmoid scores, renormalised
        dict(name="route_backward_r1", op="route_backward", T=4096, E=256, k=8, score="sigmoid", renormalize=True,
             scale=2.5, out="bf16"),
        # every tensor of a small layer, odd sizes among them: fp32 states, bf16 weights with fp32 masters
        dict(name="adamw_small_layer", op="adamw", tensors=24, largest=65536, states=32, param="bf16", master=True,
             grad="bf16"),
        # weights of a few V2-Lite-shaped experts: 8-bit states, bf16 weights rounded stochastically
        dict(name="adamw_experts_8bit", op="adamw", tensors=17, largest=5767168, states=8, param="bf16", master=False,
             grad="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "swiglu", "swiglu_backward", "combine_backward", "route_backward", "adamw"])
    if op in ("gemm", "swiglu", "swiglu_backward"):
        dt = "f32" if rng.random() < 0.2 else "bf16"
        step = 4 if dt == "f32" else 8                     # rows start on 16 bytes
        top = 512 if dt == "f32" else 2816
        case = dict(op=op, rows=_log_int(rng, 1, 1024 if dt == "f32" else 36006), experts=rng.choice([0, 1, 3, 8, 37, 64]),
                    skew=rng.choice([0.0, 0.6, 1.2]), spare=rng.choice([0, 0, 1, 70]), dt=dt)
        one, two = step * _log_int(rng, 1, top // step), step * _log_int(rng, 1, 2048 // step if dt == "bf16" else 128)
        if op == "gemm":
            return dict(case, kind=rng.choice(["nt", "nn", "tn"]), N=one, K=two,
                        out="f32" if dt == "f32" else rng.choice(["bf16", "f32"]), accumulate=rng.random() < 0.4)
        return dict(case, H=two, I=max(step, one // (2 * step) * step))
    if op == "combine_backward":
        dt = rng.choice(["bf16", "bf16", "f32"])
        step = 4 if dt == "f32" else 8
        return dict(op=op, T=_log_int(rng, 1, 8192), H=step * _log_int(rng, 1, 2048 // step), k=rng.randint(1, 8),
                    local=rng.choice([1.0, 0.5, 0.125]), dt=dt)
    if op == "route_backward":
        E = rng.randint(1, 256)
        return dict(op=op, T=_log_int(rng, 1, 8192), E=E, k=rng.randint(1, min(E, 16)),
                    score=rng.choice(["softmax", "sigmoid"]), renormalize=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), out=rng.choice(["bf16", "f32"]))
    param = rng.choice(["bf16", "f32"])
    return dict(op=op, tensors=_log_int(rng, 1, 100), largest=_log_int(rng, 1, 1 << 20), states=rng.choice([8, 32]),
                param=param, master=param == "bf16" and rng.random() < 0.5, grad=rng.choice(["bf16", "f32"]))


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _counts(case, seed):
    """Rows of each expert: independent draws from a Zipf-like popularity (skew 0: uniform)."""
    E, rows = case["experts"], case["rows"]
    if E == 0:
        return None
    g = torch.Generator().manual_seed(seed * 7 + 1)
    p = torch.arange(1, E + 1, dtype=torch.float64).pow(-case["skew"])[torch.randperm(E, generator=g)]
    if case["skew"] > 1 and E > 1:
        p[int(p.argmin())] = 0.0
    ids = torch.multinomial(p, rows, replacement=True, generator=g)
    return torch.bincount(ids, minlength=E)


def _prepare_rows(case, seed):
    cnt = _counts(case, seed)
    s = dict(case)
    s["M"], s["cap"] = case["rows"], case["rows"] + case["spare"] if cnt is not None else case["rows"]
    if cnt is None:
        s["offsets"], s["counts"] = None, [case["rows"]]
    else:
        off = torch.zeros(case["experts"] + 1, dtype=torch.int32)
        off[1:] = cnt.cumsum(0)
        s["offsets"], s["counts"] = off.to(DEV), cnt.tolist()
    s["E"] = len(s["counts"])
    return s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]

    def normal(*shape, std=1.0, dt=torch.float32):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dt)

    if op in ("gemm", "swiglu", "swiglu_backward"):
        s = _prepare_rows(case, seed)
        dt, E, cap = DT[case["dt"]], s["E"], s["cap"]
        if op == "gemm":
            N, K = case["N"], case["K"]
            if case["kind"] == "tn":
                s["a"], s["b"], cshape = normal(cap, N, dt=dt), normal(cap, K, dt=dt), (E, N, K)
            else:
                s["a"], cshape = normal(cap, K, dt=dt), (cap, N)
                s["b"] = normal(E, *((N, K) if case["kind"] == "nt" else (K, N)), std=K ** -0.5, dt=dt)
            s["c"] = normal(*cshape, dt=DT[case["out"]]) if case["accumulate"] else torch.zeros(cshape, dtype=DT[case["out"]], device=DEV)
        elif op == "swiglu":
            H, I = case["H"], case["I"]
            s["x"], s["w13"] = normal(cap, H, dt=dt), normal(E, 2 * I, H, std=H ** -0.5, dt=dt)
            s["gu"], s["h"] = (torch.zeros(cap, w, dtype=dt, device=DEV) for w in (2 * I, I))
        else:
            H, I = case["H"], case["I"]
            s["dy"], s["w2"] = normal(cap, H, dt=dt), normal(E, H, I, std=H ** -0.5, dt=dt)
            s["gu"], s["dgu"] = normal(cap, 2 * I, dt=dt), torch.zeros(cap, 2 * I, dtype=dt, device=DEV)
        return s
    if op == "combine_backward":
        T, H, k, dt = case["T"], case["H"], case["k"], DT[case["dt"]]
        local = torch.rand(T * k, generator=g, device=DEV) < case["local"]
        order = torch.randperm(T * k, generator=g, device=DEV)
        pos = torch.full((T * k,), -1, dtype=torch.int64, device=DEV)
        mine = order[local[order]]
        pos[mine] = torch.arange(mine.numel(), device=DEV)
        return dict(case, dout=normal(T, H, dt=dt), y=normal(T * k, H, dt=dt), inv=pos.to(torch.int32),
                    w=torch.rand(T, k, generator=g, device=DEV), dy=torch.zeros(T * k, H, dtype=dt, device=DEV),
                    dw=torch.empty(T, k, device=DEV))
    if op == "route_backward":
        T, E, k = case["T"], case["E"], case["k"]
        logits = normal(T, E)
        ids = torch.topk(logits + 0.5 * normal(T, E), k, dim=1).indices.to(torch.int32)
        return dict(case, logits=logits, ids=ids, dw=normal(T, k),
                    dlogits=torch.empty(T, E, dtype=DT[case["out"]], device=DEV))
    sizes = _sizes(case)
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + (n + 127) // 128 * 128)        # each tensor starts a block of 128
    n = starts[-1]
    seg = torch.zeros(n, dtype=torch.bool, device=DEV)
    for a, m in zip(starts, sizes):
        seg[a:a + m] = True
    p32 = normal(n, std=0.02) * seg
    s = dict(case, sizes=sizes, starts=starts, step=torch.full((1,), 99, dtype=torch.int32, device=DEV),
             grad_scale=torch.full((1,), 0.5, device=DEV),
             p=p32.to(DT[case["param"]]), g=(normal(n, std=0.01) * seg).to(DT[case["grad"]]),
             master=p32 if case["master"] else None)
    m, r = normal(n, std=0.003) * seg, (normal(n, std=0.01).abs() + 1e-4) * seg
    if case["states"] == 8:
        s["m"], s["m_scale"] = _encode(m)
        s["v"], s["v_scale"] = _encode(r)
    else:
        s["m"], s["v"], s["m_scale"], s["v_scale"] = m, r * r, None, None
    return s


def _sizes(case):
    """Sizes of the tensors: the largest, then smaller ones, odd ones among them."""
    n, sizes = case["largest"], []
    for i in range(case["tensors"]):
        sizes.append(max(1, (n, n // 2, n // 7 + 1, n // 64, n, n // 2, n // 1001 + 3, 1)[i % 8]))
    return sizes


# --------------------------------------------------------------------------- plain forms

HP = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, seed=1234)


def _pow2(e):
    return ((e.int() + 127) << 23).view(torch.float32)


def _block_exponent(b):
    """The smallest e >= -127 with max |b| <= 448 * 2^e, of each row: 448 = 1.75 * 2^8."""
    bits = b.abs().amax(1).view(torch.int32)
    return ((bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(-127, 127)


def _encode(x):
    """Round to nearest: [n] -> E4M3 codes [n] and E8M0 bytes [n / 128]."""
    b = x.reshape(-1, 128)
    e = _block_exponent(b)
    return (b * _pow2(-e)[:, None]).to(torch.float8_e4m3fn).reshape(-1), (e + 127).to(torch.uint8)


def _mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _hashes(s):
    """Two 32-bit random numbers of each element, from (seed, step, tensor, element)."""
    sizes = torch.tensor([b - a for a, b in zip(s["starts"], s["starts"][1:])], device=DEV)
    t = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), sizes)
    i = torch.arange(s["starts"][-1], device=DEV) - torch.tensor(s["starts"][:-1], device=DEV)[t]
    key = _mix((_mix((HP["seed"] + 0x9E3779B9 * s["step"].long()) & 0xFFFFFFFF) + 0x85EBCA77 * t) & 0xFFFFFFFF)
    one = _mix((i & 0xFFFFFFFF) ^ key)
    return one, _mix((one + 0x9E3779B9) & 0xFFFFFFFF)


def _requantize(x, rand, keep):
    """Stochastic rounding of the magnitudes to E4M3 in blocks of 128: rand has 20 bits; keep: no nonzero value
    becomes zero."""
    b = x.reshape(-1, 128)
    e = _block_exponent(b)
    y = (b.abs() * _pow2(-e)[:, None]).reshape(-1)
    normal = ((y.view(torch.int32).long() + rand) >> 20) - 960
    small = ((y * 2.0 ** 29).to(torch.int64) + rand) >> 20
    code = torch.where(y < 2.0 ** -6, small, normal)
    if keep:
        code = torch.where(y > 0, code.clamp(min=1), code)
    code = code + torch.where(torch.signbit(x), 128, 0)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _decode(codes, scale):
    e = scale.int() - 127
    return (codes.float().reshape(-1, 128) * _pow2(e // 2)[:, None] * _pow2(e - e // 2)[:, None]).reshape(-1)


def _plain_adamw(s):
    s["step"].add_(1)
    t = s["step"].double()
    lr, b1, b2 = HP["lr"], HP["beta1"], HP["beta2"]
    step_size = (lr / (1.0 - torch.pow(torch.full_like(t, b1), t))).float()
    rbc2 = (1.0 / torch.sqrt(1.0 - torch.pow(torch.full_like(t, b2), t))).float()
    eight = s["states"] == 8
    rounds = s["param"] == "bf16" and s["master"] is None         # stochastically
    one, two = _hashes(s) if eight or rounds else (None, None)
    g = s["g"].float() * s["grad_scale"]
    m = _decode(s["m"], s["m_scale"]) if eight else s["m"]
    v = _decode(s["v"], s["v_scale"]).square() if eight else s["v"]
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * (1.0 - b2)) * g
    root = torch.sqrt(v)
    p = s["master"] if s["master"] is not None else s["p"].float()
    p = p * (1.0 - lr * HP["weight_decay"]) - step_size * (m / (root * rbc2 + HP["eps"]))
    if s["master"] is not None:
        s["master"].copy_(p)
        s["p"].copy_(p)
    elif not rounds:
        s["p"].copy_(p)
    else:
        r = ((one & 0xFFF) << 4) | (two & 0xF)
        up = p.view(torch.int32).long() + r
        s["p"].copy_((up >> 16 << 16).to(torch.int32).view(torch.float32))
    if eight:
        for name, x, rand, keep in (("m", m, one >> 12, False), ("v", root, two >> 12, True)):
            codes, scale = _requantize(x, rand, keep)
            s[name].copy_(codes)
            s[name + "_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)


def _adamw_out(s):
    out = dict(p=s["p"], m=s["m"], v=s["v"])
    if s["states"] == 8:      # powers of two: a block's values are its codes' values times its scale
        out["m_scale"], out["v_scale"] = (s[n].view(torch.float8_e8m0fnu) for n in ("m_scale", "v_scale"))
    if s["master"] is not None:
        out["master"] = s["master"]
    return out


def _plain_groups(s):
    """(expert, first row, row behind the last) of each expert that has rows."""
    at = 0
    for e, n in enumerate(s["counts"]):
        if n:
            yield e, at, at + n
        at += n


def _plain(s):
    op = s["op"]
    if op == "gemm":
        a, b, c, kind = s["a"], s["b"], s["c"], s["kind"]
        if kind == "tn":
            if not s["accumulate"]:
                c.zero_()
            for e, i, j in _plain_groups(s):
                v = a[i:j].float().t() @ b[i:j].float()
                c[e] = v + c[e] if s["accumulate"] else v
        else:
            for e, i, j in _plain_groups(s):
                w = b[e].float()
                v = a[i:j].float() @ (w.t() if kind == "nt" else w)
                c[i:j] = v + c[i:j] if s["accumulate"] else v
        return c
    if op == "swiglu":
        I = s["I"]
        for e, i, j in _plain_groups(s):
            gu = s["x"][i:j].float() @ s["w13"][e].float().t()
            s["gu"][i:j] = gu
            s["h"][i:j] = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        return dict(gu=s["gu"], h=s["h"])
    if op == "swiglu_backward":
        I = s["I"]
        for e, i, j in _plain_groups(s):
            dh = s["dy"][i:j].float() @ s["w2"][e].float()
            g, u = s["gu"][i:j, :I].float(), s["gu"][i:j, I:].float()
            sg = torch.sigmoid(g)
            s["dgu"][i:j, :I] = dh * u * sg * (1.0 + g * (1.0 - sg))
            s["dgu"][i:j, I:] = dh * g * sg
        return s["dgu"]
    if op == "combine_backward":
        T, H, k = s["T"], s["H"], s["k"]
        d = s["dout"].float()[:, None, :].expand(T, k, H)
        inv = s["inv"].long().reshape(T, k)
        here = inv >= 0
        y = s["y"][inv.clamp(min=0)].float()
        s["dw"].copy_((d * y).sum(-1) * here)
        s["dy"][inv[here]] = (d * s["w"][:, :, None])[here].to(s["dy"].dtype)
        return dict(dy=s["dy"], dw=s["dw"])
    if op == "route_backward":
        l, ids, d = s["logits"], s["ids"].long(), s["dw"] * s["scale"]
        if s["score"] == "softmax":
            e = torch.exp(l - l.amax(1, keepdim=True))
            p = e / e.sum(1, keepdim=True)
        else:
            p = torch.sigmoid(l)
        q = p.gather(1, ids)
        if s["renormalize"]:
            tot = q.sum(1, keepdim=True)
            d = (d - (d * q).sum(1, keepdim=True) / tot) / tot
        full = torch.zeros_like(l).scatter_add_(1, ids, d)
        if s["score"] == "softmax":
            dl = p * (full - (p * full).sum(1, keepdim=True)) if not s["renormalize"] else p * full
        else:
            dl = full * p * torch.sigmoid(-l)
        s["dlogits"].copy_(dl)
        return s["dlogits"]
    _plain_adamw(s)
    return _adamw_out(s)


# --------------------------------------------------------------------------- the library's calls

def _own(s):
    B = _binding()
    op = s["op"]
    if op == "gemm":
        if "ws" not in s:        # a caller keeps its workspace
            n = B.moe_grouped_gemm_workspace_size(s["kind"], s["a"], s["b"], s["offsets"], s["c"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        B.moe_grouped_gemm(s["kind"], s["a"], s["b"], s["offsets"], s["c"], s["ws"], accumulate=s["accumulate"])
        return s["c"]
    if op == "swiglu":
        B.moe_grouped_swiglu(s["x"], s["w13"], s["offsets"], s["h"], gu=s["gu"])
        return dict(gu=s["gu"], h=s["h"])
    if op == "swiglu_backward":
        B.moe_grouped_swiglu_backward(s["dy"], s["w2"], s["gu"], s["offsets"], s["dgu"])
        return s["dgu"]
    if op == "combine_backward":
        B.moe_combine_backward(s["dout"], s["y"], s["inv"], s["w"], s["dy"], s["dw"])
        return dict(dy=s["dy"], dw=s["dw"])
    if op == "route_backward":
        if "rp" not in s:
            s["rp"] = B.route_params(s["E"], s["k"], s["score"], s["renormalize"], routed_scale=s["scale"])
        B.moe_route_backward(s["logits"], s["ids"], s["dw"], s["rp"], s["dlogits"])
        return s["dlogits"]
    if "table" not in s:         # the optimizer's table of tensors, made once for the life of a model
        cut = lambda t: None if t is None else [t[a:a + n] for a, n in zip(s["starts"], s["sizes"])]
        cutb = lambda t: None if t is None else [t[a // 128:a // 128 + (n + 127) // 128] for a, n in zip(s["starts"], s["sizes"])]
        s["table"] = B.moe_adamw_table(cut(s["p"]), cut(s["g"]), cut(s["m"]), cut(s["v"]), master=cut(s["master"]),
                                       m_scale=cutb(s["m_scale"]), v_scale=cutb(s["v_scale"]))
        s["hp"] = B.adamw_params(**HP)
    s["step"].add_(1)
    B.moe_adamw_step(s["table"], s["hp"], s["step"], grad_scale=s["grad_scale"])
    return _adamw_out(s)


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------- what each case cannot do without

def work(case):
    op = case["op"]
    if op in ("gemm", "swiglu", "swiglu_backward"):
        M, E, z = case["rows"], max(1, case["experts"]), 4 if case["dt"] == "f32" else 2
        # experts with rows: one popularity is zero where the skew is over 1
        used = 1 if E == 1 else min(E - (case["skew"] > 1), M)
        if op == "gemm":
            N, K, zc = case["N"], case["K"], 4 if case["out"] == "f32" else 2
            if case["kind"] == "tn":
                moved = M * (N + K) * z + (used if case["accumulate"] else E) * N * K * zc * (2 if case["accumulate"] else 1)
            else:
                moved = M * K * z + used * N * K * z + M * N * zc * (2 if case["accumulate"] else 1)
            return dict(bytes=moved, flops=2 * M * N * K)
        H, I = case["H"], case["I"]
        if op == "swiglu":
            return dict(bytes=z * (M * H + used * 2 * I * H + M * 3 * I), flops=4 * M * H * I)
        return dict(bytes=z * (M * H + used * I * H + M * 4 * I), flops=2 * M * H * I)
    if op == "combine_backward":
        T, H, k, z = case["T"], case["H"], case["k"], 4 if case["dt"] == "f32" else 2
        M = T * k * case["local"]
        return dict(bytes=z * (T * H + 2 * M * H) + 12 * T * k, flops=3 * M * H)
    if op == "route_backward":
        T, E, k = case["T"], case["E"], case["k"]
        whole = case["score"] == "softmax"                    # every logit is read; else the chosen ones
        return dict(bytes=T * ((E if whole else k) * 4 + E * (4 if case["out"] == "f32" else 2) + 8 * k), flops=T * E * 4)
    n = sum(_sizes(case))
    p = (2 if case["param"] == "bf16" else 4) * (1 if case["master"] else 2) + (8 if case["master"] else 0)
    return dict(bytes=n * (p + (2 if case["grad"] == "bf16" else 4) + 4 * (1 if case["states"] == 8 else 4)), flops=12 * n)


# --------------------------------------------------------------------------- in 64 bits

def _random_pair(sizes, starts, step):
    """The two random numbers of each element, in 32-bit arithmetic that wraps around."""
    u = np.uint32

    def mix(x):
        x = (x ^ (x >> u(16))) * u(0x7FEB352D)
        x = (x ^ (x >> u(15))) * u(0x846CA68B)
        return x ^ (x >> u(16))

    both = np.zeros((2, starts[-1]), np.uint32)
    with np.errstate(over="ignore"):
        of_step = mix(np.array([(HP["seed"] + 0x9E3779B9 * step) % 2 ** 32], np.uint32))
        for t, (a, b) in enumerate(zip(starts, starts[1:])):
            key = mix(of_step + u(0x85EBCA77 * t % 2 ** 32))
            both[0, a:b] = mix(np.arange(b - a, dtype=np.uint32) ^ key)
            both[1, a:b] = mix(both[0, a:b] + u(0x9E3779B9))
    return (torch.from_numpy(x.astype(np.int64)).to(DEV) for x in both)


def _exact_adamw(s):
    t = int(s["step"].item()) + 1
    lr, b1, b2 = HP["lr"], HP["beta1"], HP["beta2"]
    eight = s["states"] == 8

    def held(codes, scale):
        return codes.double() * torch.repeat_interleave(torch.ldexp(torch.ones_like(scale, dtype=torch.float64), scale.int() - 127), 128)

    m0 = held(s["m"], s["m_scale"]) if eight else s["m"].double()
    v0 = held(s["v"], s["v_scale"]) ** 2 if eight else s["v"].double()
    p0 = (s["p"] if s["master"] is None else s["master"]).double()
    g = s["g"].double() * s["grad_scale"].double()
    m = b1 * m0 + (1 - b1) * g
    v = b2 * v0 + (1 - b2) * g * g
    p = p0 - lr * HP["weight_decay"] * p0 - lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + HP["eps"])
    one, two = _random_pair(s["sizes"], s["starts"], t)
    out = {}

    def stochastic(x, lowest, bits, r, width):
        """x on the grid of `bits` significant bits, no finer than 2^lowest: floor(|x| / step + r / 2^width) * step."""
        step = torch.frexp(x.abs().clamp(min=1e-300))[1] - bits
        step = torch.ldexp(torch.ones_like(x), step.clamp(min=lowest))
        return torch.sign(x) * torch.floor(x.abs() / step + r.double() / 2 ** width) * step

    if s["master"] is None and s["param"] == "bf16":
        out["p"] = stochastic(p, -133, 8, ((one % 4096) * 16) + two % 16, 16)
    else:
        out["p"] = p
    if eight:
        for name, x, r in (("m", m, one // 4096), ("v", v.sqrt(), two // 4096)):
            b = x.reshape(-1, 128)
            top = b.abs().amax(1)
            e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)).clamp(-127, 127)
            y = (b / torch.exp2(e)[:, None]).reshape(-1)
            code = stochastic(y, -9, 4, r, 20)
            if name == "v":
                code = torch.where((y > 0) & (code == 0), 2.0 ** -9, code)
            out[name], out[name + "_scale"] = code, torch.exp2(e)
    else:
        out["m"], out["v"] = m, v
    if s["master"] is not None:
        out["master"] = p
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gemm", "swiglu", "swiglu_backward"):
        bounds = [0]
        for n in s["counts"]:
            bounds.append(bounds[-1] + n)
        spans = [(e, slice(bounds[e], bounds[e + 1])) for e in range(s["E"]) if bounds[e + 1] > bounds[e]]
        if op == "gemm":
            c = s["c"].double() * (1.0 if case["accumulate"] else 0.0)
            for e, r in spans:
                a = s["a"][r].double()
                if case["kind"] == "tn":
                    c[e].addmm_(a.T.contiguous(), s["b"][r].double())
                else:
                    w = s["b"][e].double()
                    c[r].addmm_(a, w.T.contiguous() if case["kind"] == "nt" else w)
            return c
        if op == "swiglu":
            gu, h = s["gu"].double(), s["h"].double()
            for e, r in spans:
                gu[r] = torch.matmul(s["x"][r].double(), s["w13"][e].double().T.contiguous())
                gate, up = gu[r].chunk(2, dim=1)
                h[r] = gate / (1.0 + torch.exp(-gate)) * up
            return dict(gu=gu, h=h)
        dgu = s["dgu"].double()
        for e, r in spans:
            gu = s["gu"][r].double().requires_grad_(True)
            gate, up = gu.chunk(2, dim=1)
            h = gate / (1.0 + torch.exp(-gate)) * up
            dgu[r] = torch.autograd.grad(h, gu, torch.matmul(s["dy"][r].double(), s["w2"][e].double()))[0]
        return dgu
    if op == "combine_backward":
        dy, dw = s["dy"].double(), torch.zeros(case["T"], case["k"], dtype=torch.float64, device=DEV)
        inv = s["inv"].long().reshape(case["T"], case["k"])
        d = s["dout"].double()
        for j in range(case["k"]):
            t = torch.nonzero(inv[:, j] >= 0).flatten()
            rows = inv[t, j]
            dy[rows] = d[t] * s["w"][t, j, None].double()
            dw[t, j] = torch.sum(s["y"][rows].double() * d[t], dim=1)
        return dict(dy=dy, dw=dw)
    if op == "route_backward":
        l = s["logits"].double().requires_grad_(True)
        p = torch.softmax(l, 1) if case["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-l))
        w = torch.gather(p, 1, s["ids"].long())
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        return torch.autograd.grad(w * case["scale"], l, s["dw"].double())[0]
    return _exact_adamw(s)
