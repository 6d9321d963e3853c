"""What the balanced gate, the integer experts, the norms and the layer made of them allow beyond the ordinary call:
gates per token in split layers, shares of the experts, single tokens, calls side by side on two streams."""
import pytest
import torch

import block_oracle as O
from test_gpu_block_layer import _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("kind", ["token", "full"])
@pytest.mark.parametrize("cid,int8", [(5, True), (5, False), (1, False)])
def test_gates_of_all_tokens_in_a_split_layer(kind, cid, int8):
    """Each microbatch takes its own part of a gate per token or a full one."""
    from combine_dual_overlap_amd import DeviceLayer, binding as B
    cfg, inp = _inputs(cid, "f32" if cid == 1 else "bf16")
    inp["block"].update(gate=None)
    layer, T = DeviceLayer(inp, int8=int8), cfg.T
    x = inp["x"].to(DEV)
    g = torch.Generator().manual_seed(3)
    gate = torch.randn(T, 1, generator=g).to(DEV) if kind == "token" else torch.randn(T, cfg.H, generator=g).to(x.dtype).to(DEV)
    b = layer.block
    layer.block_params.post.gate = gate.data_ptr()
    layer.block_params.post.gate_kind = B.MOE_GATE_TOKEN if kind == "token" else B.MOE_GATE_FULL
    for schedule, kw in (("unsplit", {}), ("dbo", {}), ("serial", dict(split_at=1)), ("dbo_recv_hook", dict(split_at=T - 3))):
        layer.out.fill_(9)
        got = layer.run(schedule, **kw).clone()
        # by halves, each an unsplit layer of its tokens with its part of the gate
        T0 = T if schedule == "unsplit" else kw.get("split_at", (T + 1) // 2)
        want = []
        for lo, hi in ((0, T0), (T0, T)):
            if lo == hi:
                continue
            part = gate[lo:hi].clone()
            layer.block_params.post.gate = part.data_ptr()
            forced = None if layer.forced_ids is None else layer.forced_ids[lo:hi].clone()
            want.append(layer.run("unsplit", x=x[lo:hi].clone(), out=torch.empty_like(x[lo:hi]), forced_ids=forced).clone())
            torch.cuda.synchronize()
        layer.block_params.post.gate = gate.data_ptr()
        if int8 or cid == 1:
            assert torch.equal(got, torch.cat(want)), schedule
        else:
            # the bf16 experts' tiles follow the number of tokens, and with them the order of fp32 sums: a rounding of
            # h (half a step, 2^-8) moves y by up to that, three roundings (h, y_perm, out) of either side
            w = torch.cat(want).double()
            assert float((got.double() - w).norm() / w.norm()) < 6 * 2.0 ** -8, schedule
    # and the gate is applied: against the layer's sum without norm and residual
    layer.block_params.post.gate_kind, layer.block_params.post.gate = B.MOE_GATE_NONE, None
    assert not torch.equal(layer.run("unsplit"), want[0][:T] if len(want) == 1 else torch.cat(want))


@pytest.mark.parametrize("T", [1, 2, 3])
@pytest.mark.parametrize("cid", [2, 5])
def test_few_tokens(cid, T):
    """A block of one, two and three tokens: every schedule gives the bits of its parts."""
    from combine_dual_overlap_amd import DeviceLayer
    cfg, inp = _inputs(cid, shared=False)
    layer = DeviceLayer(inp, int8=True)
    x = inp["x"][:T].clone().to(DEV)
    rows = [layer.run("unsplit", x=x[t:t + 1].clone(), out=torch.empty_like(x[:1])).clone() for t in range(T)]
    for schedule in ("unsplit", "serial", "dbo", "dbo_recv_hook"):
        out = torch.full_like(x, 9)
        layer.run(schedule, x=x, out=out)
        torch.cuda.synchronize()
        # (the router's product has the same split for one token as for three)
        assert torch.equal(out, torch.cat(rows)), schedule


def test_shares_of_the_experts_add_up():
    """Two shares of a layer with a norm before it, a gate and a selection bias; the balance loss with one of them."""
    from combine_dual_overlap_amd import TrainLayer
    cfg, inp = _inputs(1, "f32")
    inp["block"].update(post_norm=None, residual=False)
    half = cfg.E // 2
    whole = TrainLayer(inp, balance_coef=0.5, bias_rate=0.25)
    shares = []
    for lo, hi, coef in ((0, half, 0.5), (half, cfg.E, 0.0)):
        part = dict(inp, cfg=cfg.replace(expert_begin=lo, expert_end=hi), w13=inp["w13"][lo:hi], w2=inp["w2"][lo:hi])
        shares.append(TrainLayer(part, balance_coef=coef, bias_rate=0.25))
    x = inp["x"].to(DEV)
    dout = torch.randn(x.shape, generator=torch.Generator().manual_seed(8)).to(DEV)
    out, outs = whole.forward(x), [s.forward(x) for s in shares]
    dx, dxs = whole.backward(dout), [s.backward(dout) for s in shares]
    # chains of six sums of at most 4096 terms, in another order: sqrt(4096) * 2^-24 of the value each
    near = lambda a, b: float((a - b).norm() / b.norm()) < 6 * 64 * 2.0 ** -24
    assert near(outs[0] + outs[1], out) and near(dxs[0] + dxs[1], dx)
    assert torch.equal(shares[0].balance_loss, whole.balance_loss)
    for name in ("pre_norm", "gate", "w_router"):
        assert near(shares[0].grads[name] + shares[1].grads[name], whole.grads[name]), name
    for name in ("w13", "w2"):
        assert near(torch.cat([s.grads[name] for s in shares]), whole.grads[name]), name
    for s in shares:
        assert torch.equal(s.load, whole.load)


def _tasks():
    """Each operator's call on buffers of its own: (run, outputs)."""
    from combine_dual_overlap_amd import binding as B
    T, H, E, k, I = 700, 512, 64, 6, 320
    g = torch.Generator(device=DEV).manual_seed(5)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=g)
    new = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=DEV)
    u8, bf, i8 = torch.uint8, torch.bfloat16, torch.int8
    rp = B.route_params(E, k, "softmax", True)
    logits, bias, load = rand(T, E), 0.01 * rand(E), torch.zeros(E, dtype=torch.int32, device=DEV)
    ids, w = new(T, k, dt=torch.int32), new(T, k)
    loss, dl, ws = new(1), new(T, E), new(B.moe_route_balance_loss_workspace_size(T, E), dt=u8)

    def gate(s):
        load.zero_()
        B.moe_route_select(logits, rp, ids, w, select_bias=bias, load=load, stream=s)
        B.moe_route_balance_loss(logits, load, rp, 0.5, loss, dl, ws, stream=s)

    x, n = rand(T, H).to(bf), T * k
    cnt, off = new(E, dt=torch.int32), new(E + 1, dt=torch.int32)
    perm, inv, xq, xs = new(n, dt=torch.int32), new(n, dt=torch.int32), new(n, H, dt=i8), new(n)
    wsd = new(max(256, B.moe_dispatch_workspace_size(T, k, E)), dt=u8)
    w13, w2 = new(E, 2 * I, H, dt=i8), new(E, H, I, dt=i8)
    s13, s2 = new(E, 2 * I), new(E, H)
    B.moe_quant_int8_rows(0.05 * rand(E, 2 * I, H), w13, s13)
    B.moe_quant_int8_rows(0.05 * rand(E, H, I), w2, s2)
    y, wsf = torch.zeros(n, H, dtype=bf, device=DEV), new(B.moe_ffn_int8_workspace_size(n, I), dt=u8)
    nw, out, nn, r1, r2 = rand(H).to(bf), new(T, H, dt=bf), new(T, H, dt=bf), new(T), new(T)
    yo, dy, dw, dg, dx = new(T, H, dt=bf), new(T, H, dt=bf), new(H), new(H), new(T, H, dt=bf)
    wsn = new(B.moe_norm_backward_workspace_size(T, H), dt=u8)

    def experts(s):
        B.moe_dispatch_int8(x, ids, E, 0, E, cnt, off, perm, inv, xq, xs, wsd, stream=s)
        B.moe_grouped_ffn_int8(xq, xs, off, w13, s13, w2, s2, y, wsf, stream=s)
        B.moe_combine_post_norm(y, inv, w, x, out, 1e-6, nw, nw, 0.5, y_out=yo, rstd=r1, next_w=nw, next_n=nn, next_rstd=r2, stream=s)
        B.moe_post_norm_backward(out, yo, dy, wsn, r1, nw, dw, nw, dg, 0.5, stream=s)
        B.moe_pre_norm_backward(nn, out, r2, nw, dx, dw, wsn, dres=dy, accumulate=True, stream=s)

    def run(s):
        with torch.cuda.stream(s):
            gate(s)
            experts(s)

    return run, [ids, w, load, loss, dl, inv, xq, xs, y, out, nn, yo, dy, dw, dg, dx]


def test_two_streams_at_once():
    """The whole chain on two streams at once, eager and captured, each with its own buffers: the bits of one alone."""
    (run_a, out_a), (run_b, out_b) = _tasks(), _tasks()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    run_a(sa)
    torch.cuda.synchronize()
    want = [t.clone() for t in out_a]
    for _ in range(10):
        run_a(sa)
        run_b(sb)
    torch.cuda.synchronize()
    for a, b, t in zip(out_a, out_b, want):
        assert torch.equal(a, t) and torch.equal(b, t)
    graphs = []
    for run, s in ((run_a, sa), (run_b, sb)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run(s)
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(3):
        for t in out_a + out_b:
            t.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, (sa, sb)):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for a, b, t in zip(out_a, out_b, want):
            assert torch.equal(a, t) and torch.equal(b, t)


def test_gate_of_as_many_slots_as_experts():
    """k = E = 16, and rows whose masks leave fewer or none."""
    from combine_dual_overlap_amd import binding as B
    T, E = 33, 16
    g = torch.Generator().manual_seed(2)
    logits, bias = torch.randn(T, E, generator=g), 0.1 * torch.randn(E, generator=g)
    logits[1, 3:] = -float("inf")
    logits[2] = -float("inf")
    logits[3] = float("nan")
    logits[4] = torch.finfo(torch.float32).min
    logits[5] = float("inf")
    rp = B.route_params(E, E, "softmax", True)
    ids, w = torch.empty(T, E, dtype=torch.int32, device=DEV), torch.empty(T, E, device=DEV)
    load = torch.zeros(E, dtype=torch.int32, device=DEV)
    B.moe_route_select(logits.to(DEV), rp, ids, w, select_bias=bias.to(DEV), load=load)
    ids, w = ids.cpu(), w.cpu()
    assert torch.equal(ids.sort(1).values, torch.arange(E, dtype=torch.int32).repeat(T, 1))      # every expert once
    order = torch.argsort(bias.double(), descending=True, stable=True).int()
    assert torch.equal(ids[1, 3:], torch.arange(3, E, dtype=torch.int32)) and (w[1, 3:] == 0).all()
    assert abs(float(w[1, :3].double().sum()) - 1) <= 3 * 2.0 ** -24
    for t in (2, 3):                          # nothing left: the lowest indices, weight 0, not in the load
        assert torch.equal(ids[t], torch.arange(E, dtype=torch.int32)) and (w[t] == 0).all()
    for t in (4, 5):                          # all the same: the bias decides
        assert torch.equal(ids[t], order) and ((w[t].double() - 1 / E).abs() <= 2.0 ** -24 / E).all()
    want = torch.full((E,), T - 3)
    want[:3] += 1
    assert torch.equal(load.cpu(), want.int())


@pytest.mark.parametrize("T,H,dt", [(5, 64, torch.float32), (300, 2048, torch.bfloat16), (9, 16384, torch.float32), (4100, 1024, torch.bfloat16)])
@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
def test_norms_in_the_place_of_their_operands(T, H, dt, kind):
    """out in res's place, dy in dout's, dx in dres's: the bits of separate tensors."""
    from combine_dual_overlap_amd import binding as B
    g = torch.Generator(device=DEV).manual_seed(T)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=g)
    y, res, d = (rand(T, H).to(dt) for _ in range(3))
    w = rand(H).to(dt)
    gate = {"none": None, "channel": rand(H).to(dt), "token": rand(T, 1), "full": rand(T, H).to(dt)}[kind]
    out, rstd = torch.empty_like(y), torch.empty(T, device=DEV)
    B.moe_post_norm(y, res, out, 1e-6, w, gate, 0.5, rstd)
    there = res.clone()
    B.moe_post_norm(y, there, there, 1e-6, w, gate, 0.5)
    assert torch.equal(there, out)
    ws = torch.empty(B.moe_norm_backward_workspace_size(T, H), dtype=torch.uint8, device=DEV)
    dgate = lambda: None if gate is None else torch.empty(gate.shape, dtype=torch.float32 if kind == "channel" else gate.dtype, device=DEV)
    dy, dw, dg = torch.empty_like(y), torch.empty(H, device=DEV), dgate()
    B.moe_post_norm_backward(d, y, dy, ws, rstd, w, dw, gate, dg, 0.5)
    there, dw2, dg2 = d.clone(), torch.empty(H, device=DEV), dgate()
    B.moe_post_norm_backward(there, y, there, ws, rstd, w, dw2, gate, dg2, 0.5)
    assert torch.equal(there, dy) and torch.equal(dw, dw2) and (gate is None or torch.equal(dg, dg2))
    dx = torch.empty_like(y)
    B.moe_pre_norm_backward(d, y, rstd, w, dx, dw, ws, dres=res)
    there = res.clone()
    B.moe_pre_norm_backward(d, y, rstd, w, there, dw2, ws, dres=there)
    assert torch.equal(there, dx) and torch.equal(dw, dw2)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H,k,E,lo,hi", [(3, 8208, 6, 8, 0, 8), (70, 4112, 4, 300, 0, 300), (3000, 4112, 3, 16, 4, 9), (1025, 2048, 8, 128, 0, 128),
                                           (130, 2048, 16, 16, 0, 16), (4100, 32, 2, 260, 2, 260), (17, 16384, 2, 4, 1, 4)])
def test_dispatch_to_integers_on_every_path(T, H, k, E, lo, hi, dt):
    """Long rows, many experts, the same expert twice in a token, ties, zeros and rows that are not finite; tile offsets."""
    from combine_dual_overlap_amd import binding as B
    g = torch.Generator().manual_seed(T + H)
    x = torch.randn(T, H, generator=g)
    x[0] = 0
    x[1, 5], x[1, 6] = 4.0, 2.0                          # 2 = 63.5 scales where 4 is the largest
    x[1].clamp_(-4, 4)
    x[2, H - 1] = float("nan")
    x = x.to(dt)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)      # any expert, also twice
    E_loc, n = hi - lo, T * k
    i32 = lambda m: torch.full((m,), -9, dtype=torch.int32, device=DEV)
    meta = [i32(E_loc), i32(E_loc + 1), i32(n), i32(n), i32(E_loc + 1)]
    ws = torch.empty(max(256, B.moe_dispatch_workspace_size(T, k, E_loc)), dtype=torch.uint8, device=DEV)
    plain = torch.zeros(n, H, dtype=dt, device=DEV)
    args = (x.to(DEV), ids.to(DEV), E, lo, hi)
    B.moe_dispatch(*args, *meta[:4], plain, ws, tile_m=32, tile_offsets=meta[4])
    want = [t.clone() for t in meta]
    for t in meta:
        t.fill_(-9)
    xq, xs = torch.full((n, H), 77, dtype=torch.int8, device=DEV), torch.full((n,), -5.0, device=DEV)
    B.moe_dispatch_int8(*args, *meta[:4], xq, xs, ws, tile_m=32, tile_offsets=meta[4])
    M = int(meta[1][-1])
    for i in (0, 1, 3, 4):
        assert torch.equal(meta[i], want[i])
    assert torch.equal(meta[2][:M], want[2][:M])
    rq, rs = O.quantize(plain[:M].cpu())
    assert torch.equal(xq[:M].cpu(), rq) and torch.equal(xs[:M].cpu().nan_to_num(-1), rs.nan_to_num(-1))
    assert (xq[M:] == 77).all() and (xs[M:] == -5).all()


def test_shared_experts_of_many_tokens():
    """From 2048 tokens on the shared experts beside integer ones are grouped products: the layer is its steps with these."""
    from combine_dual_overlap_amd import DeviceLayer, binding as B
    from test_gpu_block_layer import _composed
    cfg, inp = _inputs(2, T=2100)
    layer = DeviceLayer(inp, int8=True)
    x, T, H, b = inp["x"].to(DEV), cfg.T, cfg.H, layer.block
    got = layer.run("unsplit").clone()
    near, mid = _composed(layer, x)
    shI = layer.shared_w2.shape[1]
    h, sh = torch.empty(T, shI, dtype=x.dtype, device=DEV), torch.empty_like(x)
    B.moe_grouped_swiglu(mid["xn"], layer.shared_w13[None], None, h)
    B.moe_grouped_gemm("nt", h, layer.shared_w2[None], None, sh, torch.empty(256, dtype=torch.uint8, device=DEV))
    # the shared part is the same but for the order of fp32 sums: h and the output are rounded once each
    assert float((sh.double() - mid["sh"].double()).norm() / mid["sh"].double().norm()) < 2 * 2.0 ** -8
    assert float((got.double() - near.double()).norm() / near.double().norm()) < 2 * 2.0 ** -8
    # a split layer's microbatches have fewer: the same values again, near enough
    two = layer.run("dbo", out=torch.empty_like(x))
    torch.cuda.synchronize()
    assert float((got.double() - two.double()).norm() / two.double().norm()) < 2 * 2.0 ** -8
    # and to the bit: what is left of out without the residual and the norms is the shared part's
    layer2 = DeviceLayer({**inp, "block": None}, int8=True)
    bare, routed = layer2.run("unsplit").clone(), DeviceLayer({**inp, "block": None, "shared_w13": [], "shared_w2": []}, int8=True).run("unsplit")
    h2 = torch.empty_like(h)
    B.moe_grouped_swiglu(x, layer.shared_w13[None], None, h2)
    B.moe_grouped_gemm("nt", h2, layer.shared_w2[None], None, sh, torch.empty(256, dtype=torch.uint8, device=DEV))
    want = routed.double() + sh.double()
    # routed is rounded here and not in the layer (half a step), and the sum once more
    assert ((bare.double() - want).abs() <= 2.0 ** -8 * (routed.double().abs() + want.abs()) + 1e-30).all()
