"""The norms before and after the layer and their gradients on the GPU against their 64-bit forms."""
import math

import pytest
import torch

import block_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32


def _B():
    from combine_dual_overlap_amd import binding
    return binding


def _gate(kind, g, T, H, dt):
    return {"none": lambda: None, "channel": lambda: torch.randn(H, generator=g).to(dt),
            "token": lambda: torch.rand(T, 1, generator=g), "full": lambda: torch.randn(T, H, generator=g).to(dt)}[kind]()


def _dev(t):
    return None if t is None else t.to(DEV)


def _ok(got, want, bound, dt):
    got = got.cpu().double()
    bad = (got - want).abs() > bound + O.rounding(dt, want)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}; worst {float(((got - want).abs() / (bound + O.rounding(dt, want))).max())}"


# rows of one wave and of several, chunks that end inside a wave, the largest
SHAPES = [(1, 8, BF), (3, 4, F32), (5, 520, BF), (2, 2048, BF), (9, 1000, F32), (2500, 264, BF), (2100, 2048, BF), (2049, 1024, F32),
          (7, 7168, BF), (2, 8200, BF), (3, 16384, F32), (2, 32768, BF)]


@pytest.mark.parametrize("T,H,dt", SHAPES)
def test_pre_norm(T, H, dt):
    B = _B()
    g = torch.Generator().manual_seed(T + H)
    x, w = (torch.randn(T, H, generator=g) * 3).to(dt), torch.randn(H, generator=g).to(dt)
    x[0] = 0
    n, rstd = torch.empty(T, H, dtype=dt, device=DEV), torch.empty(T, device=DEV)
    B.moe_pre_norm(x.to(DEV), w.to(DEV), n, EPS, rstd=rstd)
    v, b, r = O.norm(x.double(), torch.zeros(T, H), w.double(), EPS)
    _ok(n, v, b, dt)
    assert ((rstd.cpu().double() - r).abs() <= O.C * r).all()
    y = x.to(DEV)
    B.moe_pre_norm(y, w.to(DEV), y, EPS)                 # in place
    assert torch.equal(y, n)


@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("T,H,dt", SHAPES)
def test_post_norm(T, H, dt, kind):
    B = _B()
    g = torch.Generator().manual_seed(T + H)
    rows = lambda: torch.randn(T, H, generator=g).to(dt)
    y, res, pw, nw = rows(), rows(), torch.randn(H, generator=g).to(dt), torch.randn(H, generator=g).to(dt)
    gate = _gate(kind, g, T, H, dt)
    for post, nxt, residual in ((True, True, True), (False, True, True), (True, False, False)):
        out, n = torch.empty(T, H, dtype=dt, device=DEV), torch.full((T, H), 9.0, dtype=dt, device=DEV)
        r1, r2 = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        B.moe_post_norm(y.to(DEV), res.to(DEV) if residual else None, out, EPS, post_w=_dev(pw) if post else None,
                        gate=_dev(gate), scale=-0.75, rstd=r1 if post else None, next_w=_dev(nw) if nxt else None,
                        next_n=n if nxt else None, next_rstd=r2 if nxt else None)
        d = O.block_out(y.double(), torch.zeros(T, H), res if residual else None, EPS, pw if post else None, gate, -0.75,
                        nw if nxt else None)
        _ok(out, d["out"], d["out_bound"], dt)
        if post:
            assert ((r1.cpu().double() - d["rstd"]).abs() <= O.C * d["rstd"]).all()
        if nxt:
            _ok(n, d["n"], d["n_bound"], dt)
        if residual:
            again = res.to(DEV)
            B.moe_post_norm(y.to(DEV), again, again, EPS, post_w=_dev(pw) if post else None, gate=_dev(gate), scale=-0.75)
            assert torch.equal(again, out)               # out in the residual's place


@pytest.mark.parametrize("T,H,dt,k,shared,local", [(1, 8, BF, 1, False, 1.0), (33, 2048, BF, 6, True, 1.0), (2600, 256, BF, 8, False, 0.5),
                                                   (40, 516, F32, 3, True, 0.3), (5, 7168, BF, 16, True, 1.0), (2050, 512, F32, 2, False, 0.0),
                                                   (2100, 2048, BF, 9, False, 0.8), (3, 20000, BF, 5, True, 1.0)])
def test_combine_post_norm(T, H, dt, k, shared, local):
    B = _B()
    g = torch.Generator().manual_seed(T + H + k)
    rows = T * k
    yp = torch.randn(rows, H, generator=g).to(dt)
    inv = torch.randperm(rows, generator=g).to(torch.int32)
    inv[torch.rand(rows, generator=g) >= local] = -1
    w, res = torch.rand(T, k, generator=g), torch.randn(T, H, generator=g).to(dt)
    sh = torch.randn(T, H, generator=g).to(dt) if shared else None
    pw, nw, gate = (torch.randn(H, generator=g).to(dt) for _ in range(3))
    out, n, yo = (torch.empty(T, H, dtype=dt, device=DEV) for _ in range(3))
    r1, r2 = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    args = (yp.to(DEV), inv.to(DEV), w.to(DEV), res.to(DEV), out, EPS)
    kw = dict(post_w=_dev(pw), gate=_dev(gate), scale=0.5, shared_out=_dev(sh), next_w=_dev(nw), next_n=n)
    B.moe_combine_post_norm(*args, **kw, y_out=yo, rstd=r1, next_rstd=r2)
    y, mag = O.combine(yp, inv, w, sh)
    d = O.block_out(y, mag, res, EPS, pw, gate, 0.5, nw)
    _ok(yo, y, O.C * mag, dt)
    _ok(out, d["out"], d["out_bound"], dt)
    _ok(n, d["n"], d["n_bound"], dt)
    # y is moe_combine's output, and the outputs do not depend on what else is asked for
    ref = torch.empty(T, H, dtype=dt, device=DEV)
    B.moe_combine(yp.to(DEV), T, k, inv.to(DEV), w.to(DEV), ref, shared_out=_dev(sh))
    _ok(ref, y, O.C * mag, dt)
    first = out.clone()
    B.moe_combine_post_norm(*args, **{**kw, "next_w": None, "next_n": None})
    assert torch.equal(out, first)


def test_rows_that_are_not_finite_stay_alone():
    B = _B()
    x = torch.randn(6, 256, device=DEV)
    want = torch.empty_like(x)
    w = torch.ones(256, device=DEV)
    B.moe_pre_norm(x, w, want, EPS)
    x[1, 3], x[4, 250] = math.nan, math.inf
    n = torch.empty_like(x)
    B.moe_pre_norm(x, w, n, EPS)
    for t in (0, 2, 3, 5):
        assert torch.equal(n[t], want[t])
    assert torch.isnan(n[1]).all() and torch.isnan(n[4, 250])
    # a token without a local expert: y = 0, out = the residual
    inv = torch.full((2 * 6,), -1, dtype=torch.int32, device=DEV)
    res, out = torch.randn(6, 256, device=DEV), torch.empty(6, 256, device=DEV)
    B.moe_combine_post_norm(x, inv, torch.ones(6, 2, device=DEV), res, out, EPS, post_w=w)
    assert torch.equal(out, res)


# ------------------------------------------------------------------ gradients

def _backward(T, H, dt, kind, post, pre, residual, accumulate, seed=0):
    B = _B()
    g = torch.Generator().manual_seed(T + H + seed)
    rows = lambda s=1.0: (torch.randn(T, H, generator=g) * s).to(dt)
    d, y = rows(), rows(2.0)
    w = torch.randn(H, generator=g).to(dt) if post else None
    gate = _gate(kind, g, T, H, dt)
    rstd = (1 / torch.sqrt((y.double() ** 2).mean(1) + EPS)).float()
    dres = rows() if residual else None
    dy = torch.empty(T, H, dtype=dt, device=DEV)
    start = torch.randn(H, generator=g)
    dw = start.to(DEV) if post else None
    shape = {"channel": (H,), "token": (T, 1), "full": (T, H)}.get(kind)
    dgate = None if shape is None else start.to(DEV) if kind == "channel" else torch.empty(
        shape, dtype=dt if kind == "full" else F32, device=DEV)
    ws = torch.empty(max(256, B.moe_norm_backward_workspace_size(T, H)), dtype=torch.uint8, device=DEV)
    if pre:
        B.moe_pre_norm_backward(d.to(DEV), y.to(DEV), rstd.to(DEV), w.to(DEV), dy, dw, ws, dres=_dev(dres), accumulate=accumulate)
    else:
        B.moe_post_norm_backward(d.to(DEV), y.to(DEV), dy, ws, rstd=rstd.to(DEV) if post else None, post_w=_dev(w), dpost_w=dw,
                                 gate=_dev(gate), dgate=dgate, scale=1.0 if pre else -0.5, accumulate=accumulate)
    ref = O.norm_backward(d, y, rstd, w, gate, kind, 1.0 if pre else -0.5, dres)
    _ok(dy, *ref["dy"], dt)
    for name, got in (("dw", dw), ("dgate", dgate)):
        if got is None:
            continue
        want, bound = ref[name]
        if accumulate and got.shape == (H,):
            want, bound = want + start.double(), bound + 2 * O.U * start.abs()
        _ok(got, want, bound, got.dtype)
    return dy, dw, dgate


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H,dt", SHAPES)
def test_pre_norm_backward(T, H, dt, residual):
    _backward(T, H, dt, "none", True, True, residual, residual)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("T,H,dt", SHAPES)
def test_post_norm_backward(T, H, dt, kind, post):
    _backward(T, H, dt, kind, post, False, False, T % 2 == 0)


def test_backward_repeats_bit_for_bit_and_without_the_sums():
    B = _B()
    a = _backward(5000, 512, BF, "channel", True, False, False, False)
    b = _backward(5000, 512, BF, "channel", True, False, False, False)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    y, d, w = (torch.randn(64, 512, device=DEV) for _ in range(3))
    w = w[0].contiguous()
    rstd = torch.rsqrt(y.square().mean(1) + EPS)
    one, two = torch.empty_like(y), d.clone()
    B.moe_pre_norm_backward(d, y, rstd, w, one, None, None)
    B.moe_pre_norm_backward(two, y, rstd, w, two, None, None)           # in dn's place
    assert torch.equal(one, two)


def test_no_tokens():
    B = _B()
    e, w = torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV)
    none = torch.empty(0, device=DEV)
    B.moe_pre_norm(e, w, e, EPS, rstd=none)
    B.moe_post_norm(e, e, torch.empty(0, 64, device=DEV), EPS, post_w=w)
    dw = torch.ones(64, device=DEV)
    B.moe_pre_norm_backward(e, e, none, w, e, dw, None, accumulate=True)
    assert (dw == 1).all()
    B.moe_pre_norm_backward(e, e, none, w, e, dw, None)
    assert (dw == 0).all()


def test_offsets_past_32_bits():
    B = _B()
    T, H = 140000, 16384
    x = torch.ones(T, H, dtype=BF, device=DEV)
    x[-2:] *= 3
    w, n, rstd = torch.full((H,), 2.0, dtype=BF, device=DEV), torch.empty_like(x), torch.empty(T, device=DEV)
    B.moe_pre_norm(x, w, n, 1e-12, rstd=rstd)
    assert (n[::1013] == 2).all() and (n[-2:] == 2).all() and abs(rstd[-1].item() - 1 / 3) < 1e-6
    # d constant: dx = 0 but for rounding of the mean; the sum of dn xh over the rows is T
    dw = torch.empty(H, device=DEV)
    ws = torch.empty(B.moe_norm_backward_workspace_size(T, H), dtype=torch.uint8, device=DEV)
    d = torch.ones(T, H, dtype=BF, device=DEV)
    B.moe_pre_norm_backward(d, x, rstd, w, n, dw, ws, dres=d)
    # dx = dres + r (q - xh mean(q xh)), q = 2, xh = 1: off by fp32 roundings of terms of magnitude 2
    assert ((n[::1013].float() - 1).abs() <= 2.0 ** -8).all() and ((n[-2:].float() - 1).abs() <= 2.0 ** -8).all()
    assert ((dw - T).abs() <= T * O.C).all()


def test_captured_block_in_a_stream():
    """Norm, combine, norm and their gradients captured once and replayed on new inputs."""
    B = _B()
    T, H, k = 300, 512, 2
    g = torch.Generator().manual_seed(11)
    new = lambda *s, dt=BF: torch.empty(s, dtype=dt, device=DEV)
    x, n, out, y, dy, dx, d = (new(T, H) for _ in range(7))
    yp, rs1, rs2 = new(T * k, H), new(T, dt=F32), new(T, dt=F32)
    inv = torch.randperm(T * k, generator=g).to(torch.int32).to(DEV)
    w = torch.rand(T, k, generator=g).to(DEV)
    w1, w2, gate = (torch.randn(H, generator=g).to(BF).to(DEV) for _ in range(3))
    dw1, dw2, dg = (new(H, dt=F32) for _ in range(3))
    ws = torch.empty(B.moe_norm_backward_workspace_size(T, H), dtype=torch.uint8, device=DEV)

    def step():
        B.moe_pre_norm(x, w1, n, EPS, rstd=rs1)
        B.moe_combine_post_norm(yp, inv, w, x, out, EPS, post_w=w2, gate=gate, scale=0.5, y_out=y, rstd=rs2)
        B.moe_post_norm_backward(d, y, dy, ws, rstd=rs2, post_w=w2, dpost_w=dw2, gate=gate, dgate=dg, scale=0.5)
        B.moe_pre_norm_backward(dy, x, rs1, w1, dx, dw1, ws, dres=d)

    outs = (n, out, y, dy, dx, dw1, dw2, dg, rs1, rs2)
    graph = torch.cuda.CUDAGraph()
    for t in (x, yp, d):
        t.normal_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (x, yp, d):
            t.normal_()
        step()
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
