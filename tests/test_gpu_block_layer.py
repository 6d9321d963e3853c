"""The layer as a block of a model: 8-bit integer experts, a selection bias and the norms, gate and residual through
dbo_moe_layer and TrainLayer."""
import pytest
import torch

import block_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(cid, dt="bf16", bias=True, block=True, shared=True, **over):
    import workloads as W
    cfg = W.get_config(cid, small=True).replace(wdt=dt, act=dt, **over)
    if not shared:
        cfg = cfg.replace(n_shared=0)
    inp = W.make_inputs(cfg, 5)
    inp["forced_ids"] = None
    g = torch.Generator().manual_seed(21)
    t = inp["x"].dtype
    if bias:
        inp["select_bias"] = torch.randn(cfg.E, generator=g) * (0.1 if cfg.score == "sigmoid" else 0.5 / cfg.E)
    if block:
        new = lambda: (1 + 0.2 * torch.randn(cfg.H, generator=g)).to(t)
        inp["block"] = dict(pre_norm=new(), post_norm=new(), gate=new(), scale=0.5, eps=1e-5)
    return cfg, inp


def _composed(layer, x):
    """The layer out of its public steps, one call each."""
    from combine_dual_overlap_amd import binding as B
    cfg, b = layer.cfg, layer.block
    T, H, E, k = x.shape[0], cfg.H, cfg.E, cfg.k
    E_loc, n = cfg.expert_end - cfg.expert_begin, T * k
    new = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=DEV)
    i32, u8, t = torch.int32, torch.uint8, x.dtype
    xn = x
    if b and b["pre_norm"] is not None:
        xn = new(T, H, dt=t)
        B.moe_pre_norm(x, b["pre_norm"], xn, b["eps"])
    ids, w = new(T, k, dt=i32), new(T, k)
    ws = new(max(256, B.moe_route_workspace_size(T, H, E)), dt=u8)
    if layer.select_bias is not None:
        B.moe_route_balanced(xn, layer.w_router, layer.route, ids, w, ws, select_bias=layer.select_bias, logit_bias=layer.logit_bias)
    else:
        B.moe_route_topk(xn, layer.w_router, layer.route, ids, w, ws, logit_bias=layer.logit_bias)
    cnt, off, perm, inv = new(E_loc, dt=i32), new(E_loc + 1, dt=i32), new(n, dt=i32), new(n, dt=i32)
    ws = new(max(256, B.moe_dispatch_workspace_size(T, k, E_loc)), dt=u8)
    y = new(n, H, dt=t)
    xq, xs = new(n, H, dt=torch.int8), new(n)
    B.moe_dispatch_int8(xn, ids, E, cfg.expert_begin, cfg.expert_end, cnt, off, perm, inv, xq, xs, ws)
    B.moe_grouped_ffn_int8(xq, xs, off, layer.w13, layer.w13_scale, layer.w2, layer.w2_scale, y,
                           new(B.moe_ffn_int8_workspace_size(n, cfg.I), dt=u8))
    sh = None
    if layer.shared_w13 is not None:
        sh, shI = new(T, H, dt=t), layer.shared_w2.shape[1]
        # (the layer's own choice of tiles for these: the order of the fp32 sums is the tile's)
        tiles = lambda bm: -(-T // bm) * -(-shI // 64)
        tile = 128 if tiles(128) >= 512 else 64 if tiles(64) >= 256 else 32
        B.moe_grouped_ffn(xn, shI, None, 1, layer.shared_w13, layer.shared_w2, sh, new(B.moe_ffn_workspace_size(T, shI, B.MOE_BF16), dt=u8),
                          tile_m=tile)
    out = new(T, H, dt=t)
    if b:
        B.moe_combine_post_norm(y, inv, w, x if b["residual"] else None, out, b["eps"], b["post_norm"], b["gate"], b["scale"], shared_out=sh)
    else:
        B.moe_combine(y, T, k, inv, w, out, shared_out=sh)
    return out, dict(ids=ids, w=w, xn=xn, sh=sh)


@pytest.mark.parametrize("cid,bias,block", [(2, True, True), (3, False, True), (5, True, False), (4, True, "share")])
def test_int8_layer_is_its_steps(cid, bias, block):
    """Integer sums are exact: every schedule and split gives the bits of the separate calls."""
    from combine_dual_overlap_amd import DeviceLayer
    cfg, inp = _inputs(cid, bias=bias, block=bool(block))
    if block == "share":
        inp["block"].update(post_norm=None, residual=False)
    layer = DeviceLayer(inp, int8=True)
    x = inp["x"].to(DEV)
    layer.run("unsplit")
    torch.cuda.synchronize()
    if layer.shared_w13 is None:
        whole, _ = _composed(layer, x)
        for schedule, kw in (("unsplit", {}), ("serial", {}), ("dbo", {}), ("dbo", dict(split_at=1)), ("dbo_recv_hook", {}),
                             ("dbo", dict(comm_cu_budget=8)), ("dbo_late_event", {})):
            # (the router's product is split by the number of tokens, so its sums are those of the microbatch)
            T0 = kw.get("split_at", (cfg.T + 1) // 2)
            want = whole if schedule == "unsplit" else torch.cat([_composed(layer, x[:T0].contiguous())[0],
                                                                  _composed(layer, x[T0:].contiguous())[0]])
            layer.out.fill_(9)
            got = layer.run(schedule, **kw)
            torch.cuda.synchronize()
            assert torch.equal(got, want), schedule
    else:
        want, _ = _composed(layer, x)
        assert torch.equal(layer.run("unsplit"), want)
        T0 = (cfg.T + 1) // 2
        want = torch.cat([_composed(layer, x[:T0].contiguous())[0], _composed(layer, x[T0:].contiguous())[0]])
        assert torch.equal(layer.run("dbo"), want)


def test_int8_layer_near_the_layer_in_64_bits():
    """The experts of the chosen ids in 64 bits, without quantisation: what 8 bits cost."""
    from combine_dual_overlap_amd import DeviceLayer
    cfg, inp = _inputs(5)
    layer = DeviceLayer(inp, int8=True)
    x = inp["x"].to(DEV)
    out, mid = _composed(layer, x)
    b = layer.block
    xn = mid["xn"].cpu().double()
    ids, w = mid["ids"].cpu().long(), mid["w"].cpu().double()
    y = torch.zeros(cfg.T, cfg.H, dtype=torch.float64)
    for e in range(cfg.E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        g, u = (xn[t] @ inp["w13"][e].double().T).chunk(2, dim=1)
        y.index_add_(0, t, (g * torch.sigmoid(g) * u) @ inp["w2"][e].double().T * w[t, j, None])
    want = O.block_out(y, y.abs(), inp["x"], b["eps"], b["post_norm"].cpu(), b["gate"].cpu(), b["scale"])["out"]
    # Each quantised factor is off by an error uniform in half a step, amax / 254 / sqrt(3), against values of rms amax / 4
    # (normal, 256 of them) or more: 4 / 254 / 1.73 < 1 % each; four such factors (x, w13, h, w2; h's tails are heavier:
    # twice that), g and u both: 1 % * sqrt(2 * 2 + 1 + 4) = 3 % of y's part, and the residual is exact.
    part = want - inp["x"].double()
    rel = float((out.cpu().double() - want).norm() / part.norm())
    assert rel < 0.03, rel


def test_block_around_bf16_experts():
    """Norms, gate, residual and selection bias around the layer's other paths; forced ids come before the bias."""
    from combine_dual_overlap_amd import DeviceLayer, binding as B
    cfg, inp = _inputs(5)
    layer = DeviceLayer(inp)
    bare = DeviceLayer({**{k: v for k, v in inp.items() if k not in ("block", "select_bias")}})
    x, b = inp["x"].to(DEV), layer.block
    xn = torch.empty_like(x)
    B.moe_pre_norm(x, b["pre_norm"], xn, b["eps"])
    forced = torch.argsort(torch.rand(cfg.T, cfg.E, generator=torch.Generator().manual_seed(1)), 1)[:, :cfg.k].to(torch.int32).contiguous().to(DEV)
    y = bare.run("dbo", x=xn, forced_ids=forced).clone()
    got = layer.run("dbo", forced_ids=forced)
    want = O.block_out(y.cpu().double(), y.cpu().abs() * 2.0 ** -8 / O.C, inp["x"], b["eps"], b["post_norm"].cpu(), b["gate"].cpu(), b["scale"])
    # y of the bare layer is rounded to bf16 (half a step, in the magnitude above); the block's is not
    assert ((got.cpu().double() - want["out"]).abs() <= want["out_bound"] + O.rounding(torch.bfloat16, want["out"])).all()
    # without forced ids the bias decides: the layer at the ids of the balanced gate
    ids, w = torch.empty(cfg.T, cfg.k, dtype=torch.int32, device=DEV), torch.empty(cfg.T, cfg.k, device=DEV)
    ws = torch.empty(max(256, B.moe_route_workspace_size(cfg.T, cfg.H, cfg.E)), dtype=torch.uint8, device=DEV)
    B.moe_route_balanced(xn, layer.w_router, layer.route, ids, w, ws, select_bias=layer.select_bias, logit_bias=layer.logit_bias)
    one = layer.run("unsplit").clone()
    view = layer.view(0, "topk_ids", torch.int32, (cfg.T, cfg.k))
    assert torch.equal(view, ids)
    two = layer.run("unsplit", forced_ids=ids)
    # the weights of forced ids are computed in fp32, the gate's in 64 bits: a few half steps of fp32 apart
    assert (one.float() - two.float()).abs().max() <= 2.0 ** -7 * one.float().abs().max()


def test_int8_block_in_a_graph():
    from combine_dual_overlap_amd import DeviceLayer
    cfg, inp = _inputs(2)
    layer = DeviceLayer(inp, int8=True)
    x = inp["x"].to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.run("dbo", x=x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run("dbo", x=x)
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)))
        want = layer.run("dbo", x=x, out=torch.empty_like(x)).clone()
        layer.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.out, want)


# ------------------------------------------------------------------ training

def _block64(cfg, inp, W, b, x, ids, load, coef):
    """(out, balance loss) in 64 bits at given ids."""
    def norm(v, w):
        return v * torch.rsqrt((v * v).mean(1, keepdim=True) + b["eps"]) * w

    xn = norm(x, W["pre_norm"]) if "pre_norm" in W else x
    logits = xn @ W["w_router"][0].T
    if inp["logit_bias"] is not None:
        logits = logits + inp["logit_bias"].double()
    p = torch.softmax(logits, 1) if cfg.score == "softmax" else torch.sigmoid(logits)
    w = p.gather(1, ids)
    if cfg.renormalize:
        w = w / w.sum(1, keepdim=True)
    w = w * cfg.routed_scale
    y = torch.zeros_like(x)

    def swiglu(z, w13, w2):
        g, u = (z @ w13.T).chunk(2, dim=1)
        return (g * torch.sigmoid(g) * u) @ w2.T

    for e in range(cfg.E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            y = y.index_add(0, t, swiglu(xn[t], W["w13"][e], W["w2"][e]) * w[t, j, None])
    if "shared_w13" in W:
        y = y + swiglu(xn, W["shared_w13"][0], W["shared_w2"][0])
    z = norm(y, W["post_norm"]) if "post_norm" in W else y
    z = z * W["gate"] if "gate" in W else z
    out = b["scale"] * z + (x if b["residual"] else 0)
    q = p / p.sum(1, keepdim=True)
    return out, coef * cfg.E * (load.double() / load.sum() * q.mean(0)).sum()


@pytest.mark.parametrize("cid,dt,parts", [(1, "f32", "all"), (1, "f32", "no pre"), (1, "f32", "no post"), (1, "f32", "residual"), (2, "bf16", "all"),
                                          (5, "bf16", "all")])
def test_train_block_gradients(cid, dt, parts):
    """Forward, backward twice (gradients add up), against 64-bit autograd at the same experts."""
    from combine_dual_overlap_amd import TrainLayer
    cfg, inp = _inputs(cid, dt)
    b = inp["block"]
    b["residual"] = True
    if parts == "no pre":
        b["pre_norm"] = None
    if parts == "no post":
        b.update(post_norm=None, residual=False)
    if parts == "residual":
        b.update(pre_norm=None, post_norm=None, gate=None)
    coef = 0.5
    layer = TrainLayer(inp, balance_coef=coef)
    x = inp["x"].to(DEV)
    dout = torch.randn(x.shape, generator=torch.Generator().manual_seed(8)).to(x.dtype)
    out = layer.forward(x).clone()
    ids = layer.buf["ids"][:cfg.T].cpu().long()
    assert torch.equal(layer.load.cpu(), torch.bincount(ids.flatten(), minlength=cfg.E).int())
    dx = layer.backward(dout.to(DEV)).clone()
    loss = layer.balance_loss.item()
    first = {n: t.clone() for n, t in layer.grads.items()}
    layer.forward(x)
    layer.backward(dout.to(DEV))
    for n, t in layer.grads.items():
        assert (t - 2 * first[n]).abs().max() <= 2.0 ** -20 * t.abs().max(), n
    W = {n: t.cpu().double().requires_grad_(True) for n, t in layer.weights.items()}
    x64 = inp["x"].double().requires_grad_(True)
    ref, ref_loss = _block64(cfg, inp, W, b, x64, ids, layer.load.cpu(), coef)
    grads = torch.autograd.grad((ref * dout.double()).sum() + ref_loss, [x64, *W.values()])
    rel = lambda a, r: float((a.cpu().double() - r).norm() / r.norm())
    # fp32: six products of at most 512 terms, each off by at most terms * 2^-24: 2e-4.  bf16: at most twelve stored
    # intermediates on a path, each off by 2^-8 / sqrt(3) of its value: 0.8 %, and the differences in the norms' and the
    # gate's gradients stand for a factor of 2.5
    tol = 2e-4 if dt == "f32" else 2e-2
    assert rel(out, ref.detach()) < tol
    assert abs(loss - ref_loss.item()) <= tol * ref_loss.item()
    assert rel(dx, grads[0]) < tol
    for n, r in zip(W, grads[1:]):
        assert rel(first[n], r) < tol, n


@pytest.mark.parametrize("states,master", [("f32", True), ("fp8", False)])
def test_train_block_steps(states, master):
    """A step moves every weight, the norms without decay, and the bias towards the experts with fewer tokens."""
    from combine_dual_overlap_amd import TrainLayer
    cfg, inp = _inputs(2)
    layer = TrainLayer(inp, states=states, master=master, lr=1e-2, weight_decay=0.5, balance_coef=0.01, bias_rate=0.125)
    x = inp["x"].to(DEV)
    dout = torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).to(x.dtype).to(DEV)
    old = {n: w.float().clone() for n, w in layer.weights.items()}
    bias = layer.select_bias.clone()
    layer.forward(x)
    load = layer.load.clone()
    layer.backward(dout)
    layer.forward(x)
    layer.backward(dout)
    gr = {n: g.clone() for n, g in layer.grads.items()}
    layer.step()
    want = bias + 0.125 * torch.sign(load.float().mean() - load.float())
    assert torch.equal(layer.select_bias, want) and layer.load_sum.abs().sum() == 0
    for n in ("pre_norm", "post_norm", "gate"):
        # the first step: lr * sign(gradient) (eps apart), and no decay; bf16 steps at 1 are 2^-7 wide
        d = layer.weights[n].float() - old[n]
        sure = gr[n].abs() > 1e-4
        assert ((d + 1e-2 * torch.sign(gr[n])).abs() <= 2.0 ** -7 * old[n].abs() + 1e-4)[sure].all(), n
    for n, w in layer.weights.items():
        assert not torch.equal(w.float(), old[n]), n
    with pytest.raises(RuntimeError):
        layer.step()


def test_train_block_step_in_a_graph():
    from combine_dual_overlap_amd import TrainLayer
    def make():
        cfg, inp = _inputs(2)
        layer = TrainLayer(inp, balance_coef=0.01, bias_rate=0.01, lr=1e-3)
        return layer, inp["x"].to(DEV), torch.randn(inp["x"].shape, generator=torch.Generator().manual_seed(4)).to(inp["x"].dtype).to(DEV)

    eager, x, dout = make()
    graphed, xg, dg = make()

    def step(layer, x, dout):
        layer.forward(x)
        dx = layer.backward(dout)
        layer.step()
        return dx

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(graphed, xg, dg)
    torch.cuda.synchronize()
    step(eager, x, dout)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dxg = step(graphed, xg, dg)
    for i in range(3):
        t = torch.randn(x.shape, generator=torch.Generator().manual_seed(30 + i)).to(x.dtype)
        x.copy_(t)
        xg.copy_(t)
        dx = step(eager, x, dout)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, dxg)
        for n in eager.weights:
            assert torch.equal(eager.weights[n], graphed.weights[n]), (i, n)
        assert torch.equal(eager.select_bias, graphed.select_bias) and torch.equal(eager.balance_loss, graphed.balance_loss)
