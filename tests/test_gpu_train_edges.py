"""Corners of the training operators on the GPU: second moments below fp32's normal range, gradients that are not
finite, experts without rows, refused and captured training steps, fp32 tiles and split reductions.

Tolerances count roundings as the other tests of these operators do: `check` is theirs.
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_train import (BF, E4M3, F32, TALL, _B, _decode, _layer_inputs, _ref_rows, _sigmoid, _swiglu_bwd, check,
                            offsets_of, rnd, spans)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ AdamW far from 1

def _update(p0, m1, v1, t, b1, b2, eps):
    """The parameter after a step of lr 1 without decay, from the new moments, in 64 bits."""
    return p0 - m1 / (1 - b1 ** t) / (np.sqrt(v1 / (1 - b2 ** t)) + eps)


@pytest.mark.parametrize("beta2", [0.95, 0.999])
@pytest.mark.parametrize("master", [False, True], ids=["f32", "master"])
def test_adamw_second_moment_below_the_normal_range(master, beta2):
    """fp32 states whose v is denormal: the update still divides by its root, not by eps alone."""
    B = _B()
    n, eps = 4099, 1e-30
    g = torch.Generator().manual_seed(21)
    gr = (10.0 ** (torch.rand(n, generator=g, dtype=torch.float64) * 8 - 22) * torch.sign(rnd(g, n))).float().cuda()
    gr[5] = 0.0
    ma = torch.zeros(n, device="cuda")
    p = torch.zeros(n, dtype=BF, device="cuda") if master else ma
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    table = B.moe_adamw_table([p], [gr], [m], [v], master=[ma] if master else None)
    hp = B.adamw_params(lr=1.0, beta2=beta2, eps=eps, weight_decay=0.0)
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    gd = gr.double().cpu().numpy()
    u = 2.0 ** -24
    for t in (1, 2, 3):
        p0, m0, v0 = (x.double().cpu().numpy() for x in (ma, m, v))
        step.add_(1)
        B.moe_adamw_step(table, hp, step)
        m1, v1 = 0.9 * m0 + 0.1 * gd, beta2 * v0 + (1 - beta2) * gd * gd
        # m: 4 roundings; v: 4 roundings, and three of them may be of denormals, half of 2^-149 each.  The update lies
        # between those of the smallest and the largest root, with 12 roundings of its own.
        em, ev = 4 * u * (0.9 * np.abs(m0) + 0.1 * np.abs(gd)) + 1e-44, 4 * u * v1 + 1.5 * 2.0 ** -149
        ends = [_update(0, m1 + i * em, np.maximum(v1 + j * ev, 0), t, 0.9, beta2, eps) for i in (-1, 1) for j in (-1, 1)]
        lo, hi = p0 + np.minimum.reduce(ends), p0 + np.maximum.reduce(ends)
        slack = 3 * u * np.abs(p0) + 12 * u * np.maximum.reduce(np.abs(ends))
        got = ma.double().cpu().numpy()
        bad = (got < lo - slack) | (got > hi + slack)
        assert not bad.any(), (t, int(bad.sum()), gd[bad][:3], got[bad][:3], lo[bad][:3], hi[bad][:3])
        assert (np.abs(v.double().cpu().numpy() - v1) <= ev).all()
        assert got[5] == 0.0


@pytest.mark.parametrize("param", [F32, BF], ids=["f32", "bf16"])
def test_adamw_8bit_states_at_every_magnitude(param):
    """Blocks from 1 down to denormal gradients, and blocks that span the whole range: a nonzero second moment keeps a
    nonzero code, codes bracket the formula's values and the update divides by the root."""
    B = _B()
    blocks, eps, b2 = 46, 1.2e-38, 0.95
    n = 128 * blocks + 37
    g = torch.Generator().manual_seed(22)
    mag = 10.0 ** -(torch.arange(n) // 128).double().clamp(max=40)
    wide = 10.0 ** -(torch.rand(n, generator=g, dtype=torch.float64) * 41)
    mag = torch.where((torch.arange(n) // 128) % 4 == 3, wide, mag)
    gr = torch.zeros(n, device="cuda")
    p = torch.zeros(n, dtype=param, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros((n + 127) // 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = B.moe_adamw_table([p], [gr], [m], [v], [ms], [vs])
    hp = B.adamw_params(lr=1.0, beta2=b2, eps=eps, weight_decay=0.0)
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    u = 2.0 ** -24
    for t in (1, 2, 3):
        if t < 3:
            gr.copy_(((0.5 + torch.rand(n, generator=g)) * torch.sign(rnd(g, n)) * mag).float())
        else:
            gr.zero_()                                        # the states only decay
        gd, p0 = gr.double().cpu().numpy(), p.double().cpu().numpy()
        m0, v0 = (_decode(c.cpu().numpy(), s.cpu().numpy()) for c, s in ((m, ms), (v, vs)))
        step.add_(1)
        B.moe_adamw_step(table, hp, step)
        m1, r1 = 0.9 * m0 + 0.1 * gd, np.sqrt(b2 * v0 ** 2 + (1 - b2) * gd ** 2)
        for x, codes, scale, root in ((m1, m, ms, False), (r1, v, vs, True)):
            c, s = codes.cpu().numpy(), scale.cpu().numpy()
            top = np.array([np.abs(x[j:j + 128]).max() for j in range(0, n, 128)])
            want = np.maximum(np.ceil(np.log2(np.maximum(top, 1e-300) / 448)), -127)
            near = (np.abs(top / (448 * 2.0 ** want) - 1) < 1e-5) | (np.abs(top / (224 * 2.0 ** want) - 1) < 1e-5)
            assert ((s.astype(int) - 127 == want) | near).all(), (t, root)
            sc = np.repeat(2.0 ** (s.astype(np.float64) - 127), 128)[:n]
            # m: 4 roundings of its terms, fp32's lowest step; the root: 8 roundings, and that step (of 2^-149)
            err = 8 * u * (0.9 * np.abs(m0) + 0.1 * np.abs(gd) if not root else r1) + 2.0 ** -148
            val = np.abs(_decode(c, s))
            lo = E4M3[np.searchsorted(E4M3, np.maximum(np.abs(x) - err, 0) / sc, side="right") - 1] * sc
            hi = E4M3[np.minimum(np.searchsorted(E4M3, (np.abs(x) + err) / sc, side="left"), 126)] * sc
            if root:
                hi = np.where(x > 0, np.maximum(hi, 2.0 ** -9 * sc), hi)
                assert ((c != 0) == (x > 0)).all(), (t, int(((c != 0) != (x > 0)).sum()), x[(c != 0) != (x > 0)][:4])
            assert ((val >= lo) & (val <= hi)).all(), (t, root)
        den = r1 / np.sqrt(1 - b2 ** t) + eps
        up = m1 / (1 - 0.9 ** t) / den
        err = (4 * u * (0.9 * np.abs(m0) + 0.1 * np.abs(gd)) + 2.0 ** -148) / (1 - 0.9 ** t) / den
        err += np.abs(up) * (16 * u + 2.0 ** -148 / den) + 3 * u * np.abs(p0)
        if param == BF:                                       # a stochastic rounding: less than one bf16 step
            err += 2.0 ** -7 * (np.abs(p0 - up) + err) + 2.0 ** -133
        bad = np.abs(p.double().cpu().numpy() - (p0 - up)) > err
        assert not bad.any(), (t, int(bad.sum()), gd[bad][:3])


@pytest.mark.parametrize("param", [F32, BF], ids=["f32", "bf16"])
def test_adamw_8bit_states_keep_what_is_not_finite(param):
    """An infinity or NaN stays in its own element, as NaN codes; the block's other elements are what they are beside
    a gradient of zero."""
    B = _B()
    n = 128 * 40 + 50
    bad = {3: math.inf, 130: math.nan, 131: -math.inf, 300: math.inf, 2047: math.nan, n - 1: -math.inf}
    bad.update({i: math.nan for i in range(512, 640)})        # a block with nothing else
    at = torch.tensor(sorted(bad))
    keep = torch.ones(n, dtype=torch.bool)
    keep[at] = False
    g = torch.Generator().manual_seed(23)
    p0 = rnd(g, n, dt=param)

    def make():
        codes = lambda k: torch.zeros(k, dtype=torch.uint8, device="cuda")
        s = dict(p=p0.cuda(), g=torch.zeros(n, device="cuda"), m=codes(n), v=codes(n), ms=codes((n + 127) // 128),
                 vs=codes((n + 127) // 128))
        s["table"] = B.moe_adamw_table([s["p"]], [s["g"]], [s["m"]], [s["v"]], [s["ms"]], [s["vs"]])
        return s

    a, b = make(), make()
    hp, step = B.adamw_params(lr=0.01), torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in (1, 2, 3):
        grad = rnd(g, n)
        clean = grad * keep                                   # zeros in b, so that its states there stay zero
        if t == 1:
            for i, x in bad.items():
                grad[i] = x
        a["g"].copy_(grad)
        b["g"].copy_(clean)
        step.add_(1)
        for s in (a, b):
            B.moe_adamw_step(s["table"], hp, step)
        for name in ("p", "m", "v"):
            assert torch.equal(a[name].cpu()[keep], b[name].cpu()[keep]), (t, name)
        assert torch.equal(a["ms"], b["ms"]) and torch.equal(a["vs"], b["vs"]), t
        assert torch.isnan(a["p"].cpu()[at]).all(), t
        for name in ("m", "v"):
            assert torch.isnan(a[name].view(torch.float8_e4m3fn).float().cpu()[at]).all(), (t, name)


# ------------------------------------------------------------------ grouped products

# tiles of 64 rows with and without a split reduction, of 128, of 256 (only where C is fp32 and experts are tall), and
# the fp32 kernel's with and without a split
@pytest.mark.parametrize("dt,N,K,counts,split", [(BF, 72, 136, [40, 0, 70, 33], False), (BF, 72, 136, [4700, 0, 0, 300], True),
                                                 (BF, 1032, 520, [0, 300, 17, 0, 1], False), (BF, 520, 1032, TALL, False),
                                                 (F32, 68, 36, [40, 0, 70, 33], False), (F32, 64, 64, [0, 4000, 0, 96], True)],
                         ids=["64", "64split", "128", "256", "f32", "f32split"])
def test_weight_gradients_leave_experts_without_rows(dt, N, K, counts, split):
    """Adding to C: an expert without rows keeps its bits, negative zeros and NaN patterns among them."""
    B = _B()
    g = torch.Generator().manual_seed(31)
    M = sum(counts)
    a, b = rnd(g, M, N, dt=dt), rnd(g, M, K, dt=dt)
    off = offsets_of(counts).cuda()
    for out in (F32, BF) if dt == BF else (F32,):
        c0 = rnd(g, len(counts), N, K, dt=out)
        bits = torch.int32 if out == F32 else torch.int16
        idle = [e for e, n in enumerate(counts) if n == 0]
        for e in idle:
            c0[e].view(-1)[0::3] = -0.0
            c0[e].view(bits).view(-1)[1::5] = 0x7fa5 << (16 if out == F32 else 0)     # a signalling NaN
        c = c0.cuda()
        ac, bc = a.cuda(), b.cuda()
        need = B.moe_grouped_gemm_workspace_size("tn", ac, bc, off, c)
        assert (need > 0) == split
        print(f"idle experts {dt} N={N} K={K} {out} ws={need}", flush=True)
        B.moe_grouped_gemm("tn", ac, bc, off, c, torch.empty(need, dtype=torch.uint8, device="cuda"), accumulate=True)
        for e in idle:
            assert torch.equal(c[e].cpu().view(bits), c0[e].view(bits)), e
        for e, r in spans(counts):
            if counts[e]:
                x, y, z = a[r].double().T, b[r].double(), c0[e].double()
                check(c[e], x @ y + z, x.abs() @ y.abs() + z.abs(), max(counts) + 32, "beside idle experts")
        # without adding: zeros
        B.moe_grouped_gemm("tn", ac, bc, off, c, torch.empty(need, dtype=torch.uint8, device="cuda"))
        for e in idle:
            assert (c[e].cpu().view(bits) == 0).all(), e


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_weight_gradients_of_no_rows_at_all(dt):
    """Row operands of length zero: zeros, or C as it was where the product is added."""
    B = _B()
    for E, off in ((1, None), (3, torch.zeros(4, dtype=torch.int32, device="cuda"))):
        a, b = torch.empty(0, 72, dtype=dt, device="cuda"), torch.empty(0, 136, dtype=dt, device="cuda")
        c = torch.full((E, 72, 136), -0.0, device="cuda")
        B.moe_grouped_gemm("tn", a, b, off, c, accumulate=True)
        assert (c.view(torch.int32) == -2 ** 31).all()
        B.moe_grouped_gemm("tn", a, b, off, c)
        assert (c.view(torch.int32) == 0).all()


# ------------------------------------------------------------------ fp32 tiles, split reductions

# rows around the 64-row tile and its second half, several tiles an expert (of equal height), one row, none
TILES = [1, 33, 0, 63, 64, 65, 129, 200, 31, 32]


@pytest.mark.parametrize("kind", ["nt", "nn"])
def test_grouped_gemm_f32_of_many_tiles(kind):
    """Enough 64 x 64 tiles that fp32 products take them."""
    B = _B()
    g = torch.Generator().manual_seed(41)
    M, off = sum(TILES), offsets_of(TILES).cuda()
    for N, K in ((1028, 100), (1092, 12)):
        for acc in (False, True):
            print(f"{kind} f32 N={N} K={K} acc={acc}", flush=True)
            a, c0 = rnd(g, M + 3, K), rnd(g, M + 3, N)
            a[M:] = math.nan
            b = rnd(g, len(TILES), *((N, K) if kind == "nt" else (K, N)))
            c = c0.cuda()
            B.moe_grouped_gemm(kind, a.cuda(), b.cuda(), off, c, accumulate=acc)
            ref, mag = _ref_rows(kind, a[:M], b, TILES)
            if acc:
                ref, mag = ref + c0[:M].double(), mag + c0[:M].double().abs()
            check(c[:M], ref, mag, K, "f32 tiles")
            assert torch.equal(c[M:].cpu(), c0[M:])


def test_grouped_swiglu_f32_of_many_tiles():
    B = _B()
    g = torch.Generator().manual_seed(42)
    M, off = sum(TILES), offsets_of(TILES).cuda()
    for I, H in ((1028, 100), (1092, 12)):
        print(f"swiglu f32 I={I} H={H}", flush=True)
        x, w13 = rnd(g, M, H), rnd(g, len(TILES), 2 * I, H, std=H ** -0.5)
        gu, h = torch.zeros(M + 2, 2 * I, device="cuda"), torch.zeros(M + 2, I, device="cuda")
        xs = torch.cat([x, torch.full((2, H), math.nan)]).cuda()
        B.moe_grouped_swiglu(xs, w13.cuda(), off, h, gu=gu)
        ref, mag = _ref_rows("nt", x, w13, TILES)
        check(gu[:M], ref, mag, H, "gu")
        gate, up, mg, mu = ref[:, :I], ref[:, I:], mag[:, :I], mag[:, I:]
        s = _sigmoid(gate)
        check(h[:M], gate * s * up, (H + 2) * (1.1 * up.abs() * mg + (gate * s).abs() * mu) + 16 * (gate * s * up).abs(), -1, "h")
        assert (gu[M:] == 0).all() and (h[M:] == 0).all()
        dy, w2, gu64 = rnd(g, M, H), rnd(g, len(TILES), H, I, std=H ** -0.5), gu[:M].cpu().double()
        dgu = torch.zeros(M + 2, 2 * I, device="cuda")
        B.moe_grouped_swiglu_backward(torch.cat([dy, torch.full((2, H), math.nan)]).cuda(), w2.cuda(), gu, off, dgu)
        dh, mag = _ref_rows("nn", dy, w2, TILES)
        gate, up = gu64[:, :I], gu64[:, I:]
        s = _sigmoid(gate)
        fg, fu = (up * s).abs() * (1 + gate.abs() * (1 - s)), (gate * s).abs()
        check(dgu[:M], _swiglu_bwd(dh, gu64, I), torch.cat([fg, fu], 1) * ((H + 2) * mag + 16 * dh.abs()).repeat(1, 2), -1, "dgu")
        assert (dgu[M:] == 0).all()


@pytest.mark.parametrize("acc", [False, True], ids=["write", "add"])
@pytest.mark.parametrize("kind,cap,N,K,dt,out", [("tn", 5000, 72, 136, BF, BF), ("nt", 33, 72, 4104, BF, BF),
                                                 ("nn", 33, 72, 4104, BF, BF), ("tn", 4096, 64, 64, F32, F32),
                                                 ("tn", 4099, 68, 132, F32, F32)])
def test_split_reductions_to_each_type(kind, cap, N, K, dt, out, acc):
    """Parts of the fp32 kernel, and joins that write bf16: rounded once, rows and experts as in the unsplit call."""
    B = _B()
    g = torch.Generator().manual_seed(43)
    for counts in (None, [cap // 3, 0, cap // 5, 1]):
        E = 1 if counts is None else 4
        if kind == "tn":
            a, b, c0 = rnd(g, cap, N, dt=dt), rnd(g, cap, K, dt=dt), rnd(g, E, N, K, dt=out)
        else:
            a, c0 = rnd(g, cap, K, dt=dt), rnd(g, cap, N, dt=out)
            b = rnd(g, E, *((N, K) if kind == "nt" else (K, N)), dt=dt)
        off = None if counts is None else offsets_of(counts).cuda()
        c, ac, bc = c0.cuda(), a.cuda(), b.cuda()
        need = B.moe_grouped_gemm_workspace_size(kind, ac, bc, off, c)
        print(f"split {kind} cap={cap} N={N} K={K} {dt} {out} acc={acc} E={E} ws={need}", flush=True)
        assert need > 0 or counts is not None
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")               # NaN patterns
        B.moe_grouped_gemm(kind, ac, bc, off, c, ws, accumulate=acc)
        z0 = c0.double() if acc else torch.zeros_like(c0, dtype=torch.float64)
        ref, mag = z0.clone(), z0.abs()
        for e, r in spans([cap] if counts is None else counts):
            if kind == "tn":
                x, y, z = a[r].double().T, b[r].double(), e
            else:
                x, y, z = a[r].double(), b[e].double().T if kind == "nt" else b[e].double(), r
            ref[z] += x @ y
            mag[z] += x.abs() @ y.abs()
        rows = len(ref) if kind == "tn" or counts is None else sum(counts)
        check(c[:rows], ref[:rows], mag[:rows], max(cap, K) + 32, "split")
        assert torch.equal(c[rows:].cpu(), c0[rows:])


# ------------------------------------------------------------------ the layer

def test_train_layer_step_that_is_refused_changes_nothing():
    """A step refused for its scalars leaves the step count, so that the next one corrects its moments as the first."""
    from combine_dual_overlap_amd import TrainLayer
    B = _B()
    cfg, inp = _layer_inputs(2, "bf16", forced=False)
    x = inp["x"].cuda()
    dout = rnd(torch.Generator().manual_seed(8), *x.shape, dt=BF).cuda()
    a, b = TrainLayer(inp), TrainLayer(inp)
    for layer in (a, b):
        layer.forward(x)
        layer.backward(dout)
    two = torch.ones(8, device="cuda")
    for kw, err in ((dict(lr_scale=torch.ones(1, dtype=torch.float64, device="cuda")), ValueError),
                    (dict(grad_scale=torch.ones(2, device="cuda")), ValueError), (dict(lr_scale=torch.ones(1)), ValueError),
                    (dict(lr_scale=two[1:2]), B.MoEError)):
        with pytest.raises(err):
            a.step(**kw)
        assert a.steps.item() == 0
    a.step()
    b.step()
    assert a.steps.item() == 1
    for n in a.weights:
        assert torch.equal(a.weights[n], b.weights[n]), n


def test_train_layer_zeroes_its_gradients():
    """What a reader of the gradients sees after zero_grad() and after step()."""
    from combine_dual_overlap_amd import TrainLayer
    _B()
    cfg, inp = _layer_inputs(2, "bf16", forced=False)
    layer = TrainLayer(inp)
    x = inp["x"].cuda()
    grads = dict(layer.grads)
    for end in (layer.zero_grad, layer.step):
        layer.forward(x)
        layer.backward(x)
        assert all((t != 0).any() for t in grads.values())
        end()
        assert all((t == 0).all() for t in grads.values())


def test_train_layer_captured_micro_steps():
    """One forward and backward captured while no gradient had been added, then replayed: every replay adds, also after
    zero_grad(), between eager calls and around eager steps; each state equals the same eager calls'."""
    from combine_dual_overlap_amd import TrainLayer
    _B()
    cfg, inp = _layer_inputs(2, "bf16", forced=False)
    g = torch.Generator().manual_seed(8)
    kw = dict(lr=2.0 ** -8)
    a, b, warm = TrainLayer(inp, **kw), TrainLayer(inp, **kw), TrainLayer(inp, **kw)
    x, dout = inp["x"].cuda(), rnd(g, *inp["x"].shape, dt=BF).cuda()

    def one(layer):
        layer.forward(x)
        layer.backward(dout)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        one(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(b)
    replay = lambda: graph.replay()
    eager = lambda: one(b)
    for calls in ((replay, replay, replay), (replay,), (eager, replay), (replay, eager, replay), (eager,)):
        for call in calls:
            x.copy_(rnd(g, *x.shape, dt=BF))
            one(a)
            call()
            torch.cuda.synchronize()
            for n in a.grads:
                assert torch.equal(a.grads[n], b.grads[n]), (n, len(calls))
        a.step()
        b.step()
        for n in a.weights:
            assert torch.equal(a.weights[n], b.weights[n]), n
    # what zero_grad() drops is gone for the replays too
    one(a)
    graph.replay()
    a.zero_grad()
    b.zero_grad()
    one(a)
    graph.replay()
    torch.cuda.synchronize()
    for n in a.grads:
        assert torch.equal(a.grads[n], b.grads[n]), n
    a.step()
    b.step()                                                  # follows a replayed backward
    for n in a.weights:
        assert torch.equal(a.weights[n], b.weights[n]), n


def test_train_layer_calls_captured_one_by_one():
    """forward(), backward() and step() in graphs of their own: two micro-steps and a step, three times, equal eager
    calls."""
    from combine_dual_overlap_amd import TrainLayer
    _B()
    cfg, inp = _layer_inputs(2, "bf16", forced=False)
    g = torch.Generator().manual_seed(8)
    kw = dict(lr=2.0 ** -8, states="fp8", master=False)
    a, b, warm = TrainLayer(inp, **kw), TrainLayer(inp, **kw), TrainLayer(inp, **kw)
    x, dout = inp["x"].cuda(), rnd(g, *inp["x"].shape, dt=BF).cuda()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        warm.forward(x)
        warm.backward(dout)
        warm.step()
    torch.cuda.synchronize()
    graphs = []
    for call in (lambda: b.forward(x), lambda: b.backward(dout), b.step):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)
    with pytest.raises(RuntimeError):
        b.backward(dout)                                      # the captured step moves the weights
    for _ in range(3):
        for _ in range(2):
            x.copy_(rnd(g, *x.shape, dt=BF))
            a.forward(x)
            a.backward(dout)
            graphs[0].replay()
            graphs[1].replay()
        a.step()
        graphs[2].replay()
        torch.cuda.synchronize()
        for n in a.weights:
            assert torch.equal(a.weights[n], b.weights[n]), n
            assert (b.grads[n] == 0).all(), n
