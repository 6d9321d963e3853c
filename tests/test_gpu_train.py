"""The training operators on the GPU against plain 64-bit implementations:
grouped matrix products, their SwiGLU epilogues, the gradients of combine and
router gate, the AdamW step, and the training layer that runs them together.

Tolerances.  A result rounded once to type t is off by at most eps(t)/2 of its
value (bf16 2^-8).  An fp32 sum of n products is off by at most
(n + 2) 2^-23 of the sum of their magnitudes: one rounding of 2^-24 for each
addition and product, twice that where the matrix unit truncates.  Both bounds
are elementwise; `bound` adds them.  expf, __expf and the divisions of the
epilogues add a few 2^-23 of their terms, counted as 16 * 2^-23.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ULP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def _B():
    import combine_dual_overlap_amd as C
    C.binding.lib()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return C.binding


def check(got, ref, mag, n, what):
    """|got - ref| within one rounding to got's type plus fp32 sums of n terms of total magnitude mag."""
    g = got.detach().cpu().double()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert torch.isfinite(g).all(), what
    # the sum's own error is rounded too, hence 1 + ULP; 1e-37: results below the normal range
    tol = ULP[got.dtype] * ref.abs() + (n + 2) * 2.0 ** -23 * mag * (1 + ULP[got.dtype]) + 1e-37
    bad = (g - ref).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst " \
        f"{float(((g - ref).abs() / tol).max()):.3g} of the bound"


def rnd(g, *shape, dt=F32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dt)


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)


def spans(counts):
    at = 0
    for e, n in enumerate(counts):
        yield e, slice(at, at + n)
        at += n


# Row counts: empty experts (first, last, all), single rows, one row more or
# less than a tile of 32, 64 or 128, more than a wave's experts, one big group.
COUNTS = {
    "one": [1], "empty": [0, 0, 0], "edges": [0, 1, 31, 32, 33, 0, 63, 65, 127, 128, 129, 0],
    "big": [300, 0, 517], "many": [(i * 7) % 5 for i in range(256)], "dense": None,
}
# (N, K): smallest, not a multiple of any tile, tile-sized, one more chunk
SIZES = {BF: [(8, 8), (136, 72), (128, 64), (264, 200)], F32: [(4, 4), (68, 36), (64, 16), (132, 100)]}


def _case(name, dt, N, K, spare, seed=0):
    counts = COUNTS[name]
    dense = counts is None
    counts = [77] if dense else counts
    g = torch.Generator().manual_seed(seed + N * 1000 + K)
    return g, counts, dense, sum(counts) + (0 if dense else spare)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("kind", ["nt", "nn"])
def test_grouped_gemm_rows(kind, name, dt):
    B = _B()
    for N, K in SIZES[dt]:
        for out, acc in ((dt, False), (F32, True), (dt, True)):
            g, counts, dense, cap = _case(name, dt, N, K, spare=3)
            print(f"{kind} {name} {dt} N={N} K={K} out={out} acc={acc}", flush=True)
            a, c0 = rnd(g, cap, K, dt=dt), rnd(g, cap, N, dt=out)
            # what lies behind the last expert is not read: it may hold anything
            a[sum(counts):] = math.nan
            b = rnd(g, len(counts), *((N, K) if kind == "nt" else (K, N)), dt=dt)
            c = c0.cuda()
            off = None if dense else offsets_of(counts).cuda()
            ac, bc = a.cuda(), b.cuda()
            ws = torch.empty(B.moe_grouped_gemm_workspace_size(kind, ac, bc, off, c), dtype=torch.uint8, device="cuda")
            B.moe_grouped_gemm(kind, ac, bc, off, c, ws, accumulate=acc)
            torch.cuda.synchronize()
            ref, mag = c0.double(), torch.zeros(cap, N, dtype=torch.float64)
            for e, r in spans(counts):
                w = b[e].double().T if kind == "nt" else b[e].double()
                ref[r] = a[r].double() @ w + (c0[r].double() if acc else 0)
                mag[r] = a[r].double().abs() @ w.abs() + (c0[r].double().abs() if acc else 0)
            M = sum(counts)
            check(c[:M], ref[:M], mag[:M], K, "product")
            assert torch.equal(c[M:].cpu(), c0[M:]), "rows behind the last expert changed"


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(COUNTS))
def test_grouped_gemm_weights(name, dt):
    B = _B()
    for N, K in SIZES[dt]:
        for out, acc in ((dt, False), (F32, True), (dt, True)):
            g, counts, dense, cap = _case(name, dt, N, K, spare=3)
            print(f"tn {name} {dt} N={N} K={K} out={out} acc={acc}", flush=True)
            a, b, c0 = rnd(g, cap, N, dt=dt), rnd(g, cap, K, dt=dt), rnd(g, len(counts), N, K, dt=out)
            a[sum(counts):], b[sum(counts):] = math.inf, math.nan
            c = c0.cuda()
            off = None if dense else offsets_of(counts).cuda()
            ac, bc = a.cuda(), b.cuda()
            ws = torch.empty(B.moe_grouped_gemm_workspace_size("tn", ac, bc, off, c), dtype=torch.uint8, device="cuda")
            B.moe_grouped_gemm("tn", ac, bc, off, c, ws, accumulate=acc)
            torch.cuda.synchronize()
            ref, mag = torch.zeros_like(c0, dtype=torch.float64), torch.zeros_like(c0, dtype=torch.float64)
            for e, r in spans(counts):
                ref[e] = a[r].double().T @ b[r].double()
                mag[e] = a[r].double().abs().T @ b[r].double().abs()
            if acc:
                ref, mag = ref + c0.double(), mag + c0.double().abs()
            check(c, ref, mag, max(counts), "weight gradient")


# Enough and large enough experts for the 256 x 256 tiles: row counts around
# one, two and several tiles, odd widths, reductions that end inside a stage.
MID = [(i * 29) % 131 for i in range(60)]                  # 128 x 128 tiles
BIG = [0, 1, 15, 16, 17, 31, 33, 255, 256, 257, 511, 513, 700, 1030, 2049] + [(i * 97) % 331 for i in range(45)]
TALL = [0, 1, 1999, 640, 513] + [450 + (i * 97) % 331 for i in range(17)]     # 256 x 256 also where TN adds to C


def _ref_rows(kind, a, b, counts):
    ref = torch.zeros(a.shape[0], b.shape[1] if kind == "nt" else b.shape[2], dtype=torch.float64)
    mag = ref.clone()
    for e, r in spans(counts):
        w = b[e].double().T if kind == "nt" else b[e].double()
        ref[r], mag[r] = a[r].double() @ w, a[r].double().abs() @ w.abs()
    return ref, mag


@pytest.mark.parametrize("N,K,counts", [(520, 72, BIG), (1032, 200, BIG), (264, 328, BIG), (648, 200, MID), (88, 136, MID), (520, 1032, TALL)],
                         ids=lambda v: "x" if isinstance(v, list) else str(v))
@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
def test_grouped_gemm_large_tiles(kind, N, K, counts):
    B = _B()
    g = torch.Generator().manual_seed(N + K)
    BIG = counts
    M, off = sum(BIG), offsets_of(BIG).cuda()
    for out, acc in ((BF, False), (F32, True)):
        print(f"{kind} large N={N} K={K} {out}", flush=True)
        a = rnd(g, M + 2, N if kind == "tn" else K, dt=BF)
        a[M:] = math.nan
        if kind == "tn":
            b, c0 = rnd(g, M + 2, K, dt=BF), rnd(g, len(BIG), N, K, dt=out)
            b[M:] = math.nan
            ref, mag = torch.zeros(c0.shape, dtype=torch.float64), torch.zeros(c0.shape, dtype=torch.float64)
            for e, r in spans(BIG):
                ref[e] = a[r].double().T @ b[r].double()
                mag[e] = a[r].double().abs().T @ b[r].double().abs()
        else:
            b, c0 = rnd(g, len(BIG), *((N, K) if kind == "nt" else (K, N)), dt=BF), rnd(g, M + 2, N, dt=out)
            ref, mag = _ref_rows(kind, a[:M], b, BIG)
        c = c0.cuda()
        ac, bc = a.cuda(), b.cuda()
        ws = torch.empty(B.moe_grouped_gemm_workspace_size(kind, ac, bc, off, c), dtype=torch.uint8, device="cuda")
        B.moe_grouped_gemm(kind, ac, bc, off, c, ws, accumulate=acc)
        n = len(ref)
        if acc:
            ref, mag = ref + c0[:n].double(), mag + c0[:n].double().abs()
        check(c[:n], ref, mag, max(BIG) if kind == "tn" else K, "large")
        if kind != "tn":
            assert torch.equal(c[M:].cpu(), c0[M:])


@pytest.mark.parametrize("I,H,counts", [(520, 72, BIG), (264, 328, BIG), (648, 200, MID), (520, 2056, BIG)],
                         ids=lambda v: "x" if isinstance(v, list) else str(v))
def test_grouped_swiglu_large_tiles(I, H, counts):
    B = _B()
    g = torch.Generator().manual_seed(I + H)
    BIG = counts
    M, off = sum(BIG), offsets_of(BIG).cuda()
    x, w13 = rnd(g, M, H, dt=BF), rnd(g, len(BIG), 2 * I, H, dt=BF, std=H ** -0.5)
    gu, h = torch.zeros(M, 2 * I, dtype=BF, device="cuda"), torch.zeros(M, I, dtype=BF, device="cuda")
    print(f"swiglu large I={I} H={H}", flush=True)
    B.moe_grouped_swiglu(x.cuda(), w13.cuda(), off, h, gu=gu)
    ref, mag = _ref_rows("nt", x, w13, BIG)
    check(gu, ref, mag, H, "gu")
    gate, up, mg, mu = ref[:, :I], ref[:, I:], mag[:, :I], mag[:, I:]
    s = _sigmoid(gate)
    check(h, gate * s * up, (H + 2) * (1.1 * up.abs() * mg + (gate * s).abs() * mu) + 16 * (gate * s * up).abs(), -1, "h")
    dy, w2, gu64 = rnd(g, M, H, dt=BF), rnd(g, len(BIG), H, I, dt=BF, std=H ** -0.5), gu.cpu().double()
    dgu = torch.zeros(M, 2 * I, dtype=BF, device="cuda")
    B.moe_grouped_swiglu_backward(dy.cuda(), w2.cuda(), gu, off, dgu)
    dh, mag = _ref_rows("nn", dy, w2, BIG)
    gate, up = gu64[:, :I], gu64[:, I:]
    s = _sigmoid(gate)
    fg, fu = (up * s).abs() * (1 + gate.abs() * (1 - s)), (gate * s).abs()
    check(dgu, _swiglu_bwd(dh, gu64, I), torch.cat([fg, fu], 1) * ((H + 2) * mag + 16 * dh.abs()).repeat(1, 2), -1, "dgu")


def test_grouped_gemm_neighbours_values_stay_out():
    """A row of infinities or NaN spoils its own expert's results only."""
    B = _B()
    counts = [40, 70, 33]
    g = torch.Generator().manual_seed(5)
    for bad in (math.inf, math.nan):
        a, b = rnd(g, 143, 136, dt=BF), rnd(g, 143, 72, dt=BF)
        a[40], b[41] = bad, bad                               # the second expert's
        c = torch.zeros(3, 136, 72, dtype=BF, device="cuda")
        B.moe_grouped_gemm("tn", a.cuda(), b.cuda(), offsets_of(counts).cuda(), c)
        for e, r in ((0, slice(0, 40)), (2, slice(110, 143))):
            check(c[e], a[r].double().T @ b[r].double(), a[r].double().abs().T @ b[r].double().abs(), 70, "neighbour")
        w, c = rnd(g, 3, 72, 136, dt=BF), torch.zeros(143, 72, dtype=BF, device="cuda")
        B.moe_grouped_gemm("nt", a.cuda(), w.cuda(), offsets_of(counts).cuda(), c)
        rows = [i for i in range(143) if i != 40]
        e_of = torch.repeat_interleave(torch.arange(3), torch.tensor(counts))
        ref = torch.stack([a[i].double() @ w[e_of[i]].double().T for i in rows])
        mag = torch.stack([a[i].double().abs() @ w[e_of[i]].double().abs().T for i in rows])
        check(c[rows], ref, mag, 136, "neighbour rows")


def test_grouped_gemm_offsets_are_kept_inside_the_rows():
    """Offsets outside [0, rows] or decreasing reach no memory outside the operands: they are cut off."""
    B = _B()
    g = torch.Generator().manual_seed(6)
    a, b = rnd(g, 50, 64, dt=BF), rnd(g, 50, 72, dt=BF)
    off = torch.tensor([-7, 20, 10, 90], dtype=torch.int32)          # rows [0, 20), none, [10, 50)
    c = torch.zeros(3, 64, 72, dtype=F32, device="cuda")
    B.moe_grouped_gemm("tn", a.cuda(), b.cuda(), off.cuda(), c)
    for e, r in ((0, slice(0, 20)), (1, slice(0, 0)), (2, slice(10, 50))):
        check(c[e], a[r].double().T @ b[r].double(), a[r].double().abs().T @ b[r].double().abs(), 40, "cut off")


# A long reduction with few output tiles is cut into parts that are joined in
# a fixed order.
@pytest.mark.parametrize("kind,cap,N,K", [("tn", 5000, 72, 136), ("nt", 33, 72, 4104), ("nn", 33, 72, 4104),
                                          ("tn", 4096, 256, 1024)])
def test_grouped_gemm_split_reduction(kind, cap, N, K):
    B = _B()
    g = torch.Generator().manual_seed(7)
    for counts in (None, [cap // 3, 0, cap // 5, 1]):
        E = 1 if counts is None else 4
        if kind == "tn":
            a, b, c0 = rnd(g, cap, N, dt=BF), rnd(g, cap, K, dt=BF), rnd(g, E, N, K)
        else:
            a, c0 = rnd(g, cap, K, dt=BF), rnd(g, cap, N)
            b = rnd(g, E, *((N, K) if kind == "nt" else (K, N)), dt=BF)
        off = None if counts is None else offsets_of(counts).cuda()
        ac, bc = a.cuda(), b.cuda()
        outs = []
        for _ in range(2):
            c = c0.cuda()
            need = B.moe_grouped_gemm_workspace_size(kind, ac, bc, off, c)
            ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")       # NaN patterns
            B.moe_grouped_gemm(kind, ac, bc, off, c, ws, accumulate=True)
            outs.append(c.cpu())
        if counts is None:
            assert need > 0, "this case is meant to be split"
        assert torch.equal(outs[0], outs[1])
        ref, mag = c0.double(), c0.double().abs()
        for e, r in spans([cap] if counts is None else counts):
            if kind == "tn":
                x, y, z = a[r].double().T, b[r].double(), e
            else:
                x, y, z = a[r].double(), b[e].double().T if kind == "nt" else b[e].double(), r
            ref[z] += x @ y
            mag[z] += x.abs() @ y.abs()
        check(outs[0], ref, mag, max(cap, K) + 32, "split")


def test_grouped_gemm_graph_replays_and_streams():
    """A split and an unsplit product captured in one graph and replayed with new inputs and new offsets between
    eager calls; then the same two products on two streams at once."""
    B = _B()
    g = torch.Generator().manual_seed(12)
    counts = [[100, 0, 333, 67], [0, 250, 1, 249], [500, 0, 0, 0]]
    a, b = rnd(g, 500, 136, dt=BF).cuda(), rnd(g, 500, 264, dt=BF).cuda()
    w = rnd(g, 4, 264, 136, dt=BF).cuda()
    x2, y2 = rnd(g, 4096, 72, dt=BF).cuda(), rnd(g, 4096, 136, dt=BF).cuda()
    off = offsets_of(counts[0]).cuda()
    c, d, e = torch.zeros(4, 136, 264, device="cuda"), torch.zeros(500, 264, dtype=BF, device="cuda"), \
        torch.zeros(1, 72, 136, device="cuda")
    need = B.moe_grouped_gemm_workspace_size("tn", x2, y2, None, e)
    assert need > 0
    ws, ws2 = (torch.zeros(need, dtype=torch.uint8, device="cuda") for _ in range(2))

    def run(c, d, e, ws):
        B.moe_grouped_gemm("tn", a, b, off, c)
        B.moe_grouped_gemm("nt", a, w, off, d)
        B.moe_grouped_gemm("tn", x2, y2, None, e, ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(c, d, e, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c, d, e, ws)
    for k in (1, 2, 0, 1):
        off.copy_(offsets_of(counts[k]))
        for t in (a, b, x2, y2):
            t.copy_(rnd(g, *t.shape, dt=BF))
        want = [torch.zeros_like(t) for t in (c, d, e)]
        run(*want, ws2)
        torch.cuda.synchronize()
        for t in (c, d, e):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for t, u in zip((c, d, e), want):
            assert torch.equal(t, u)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        got = [[torch.zeros_like(t) for t in (c, d, e)] for _ in range(2)]
        torch.cuda.synchronize()
        for s, outs, wk in ((s1, got[0], ws), (s2, got[1], ws2)):
            with torch.cuda.stream(s):
                for _ in range(5):
                    run(*outs, wk)
        torch.cuda.synchronize()
        for outs in got:
            for t, u in zip(outs, want):
                assert torch.equal(t, u)


def _sigmoid(g):
    return 1.0 / (1.0 + torch.exp(-g))


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(COUNTS))
def test_grouped_swiglu(name, dt):
    B = _B()
    for I, H in SIZES[dt]:
        g, counts, dense, cap = _case(name, dt, I, H, spare=2)
        print(f"swiglu {name} {dt} I={I} H={H}", flush=True)
        x, w13 = rnd(g, cap, H, dt=dt), rnd(g, len(counts), 2 * I, H, dt=dt, std=H ** -0.5)
        M = sum(counts)
        x[M:] = math.nan
        off = None if dense else offsets_of(counts).cuda()
        gu0, h0 = rnd(g, cap, 2 * I, dt=dt), rnd(g, cap, I, dt=dt)
        gu, h, h2 = gu0.cuda(), h0.cuda(), h0.cuda()
        B.moe_grouped_swiglu(x.cuda(), w13.cuda(), off, h, gu=gu)
        B.moe_grouped_swiglu(x.cuda(), w13.cuda(), off, h2)
        assert torch.equal(h, h2), "gu changes h"
        ref, mag = torch.zeros(cap, 2 * I, dtype=torch.float64), torch.zeros(cap, 2 * I, dtype=torch.float64)
        for e, r in spans(counts):
            ref[r] = x[r].double() @ w13[e].double().T
            mag[r] = x[r].double().abs() @ w13[e].double().abs().T
        check(gu[:M], ref[:M], mag[:M], H, "gu")
        gate, up, mg, mu = ref[:M, :I], ref[:M, I:], mag[:M, :I], mag[:M, I:]
        s = _sigmoid(gate)
        # errors of g and u pass through the derivative (at most 1.1 |u|) and silu(g); 16 for the epilogue's own
        n = (H + 2) * (1.1 * up.abs() * mg + (gate * s).abs() * mu) + 16 * (gate * s * up).abs()
        check(h[:M], gate * s * up, n, -1, "h")
        assert torch.equal(gu[M:].cpu(), gu0[M:]) and torch.equal(h[M:].cpu(), h0[M:])


def _swiglu_bwd(dh, gu, I):
    gate, up = gu[:, :I], gu[:, I:]
    s = _sigmoid(gate)
    return torch.cat([dh * up * s * (1 + gate * (1 - s)), dh * gate * s], 1)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(COUNTS))
def test_grouped_swiglu_backward(name, dt):
    B = _B()
    for I, H in SIZES[dt]:
        g, counts, dense, cap = _case(name, dt, I, H, spare=2)
        print(f"swiglu backward {name} {dt} I={I} H={H}", flush=True)
        dy, w2 = rnd(g, cap, H, dt=dt), rnd(g, len(counts), H, I, dt=dt, std=H ** -0.5)
        gu = rnd(g, cap, 2 * I, dt=dt, std=2.0)
        M = sum(counts)
        if M > 4:                                  # gates where the sigmoid is 0 or 1 in fp32
            gu[1, :I], gu[2, :I] = -200.0, 200.0
        dy[M:] = math.nan
        off = None if dense else offsets_of(counts).cuda()
        d0 = rnd(g, cap, 2 * I, dt=dt)
        dgu, inplace = d0.cuda(), gu.cuda()
        B.moe_grouped_swiglu_backward(dy.cuda(), w2.cuda(), gu.cuda(), off, dgu)
        B.moe_grouped_swiglu_backward(dy.cuda(), w2.cuda(), inplace, off, inplace)
        assert torch.equal(dgu[:M], inplace[:M])
        dh, mag = torch.zeros(cap, I, dtype=torch.float64), torch.zeros(cap, I, dtype=torch.float64)
        for e, r in spans(counts):
            dh[r] = dy[r].double() @ w2[e].double()
            mag[r] = dy[r].double().abs() @ w2[e].double().abs()
        ref = _swiglu_bwd(dh[:M], gu[:M].double(), I)
        # the factor's own terms: 1 + |g| (1 - s) bounds what cancels in it; 16 roundings of those
        gate, up = gu[:M, :I].double(), gu[:M, I:].double()
        s = _sigmoid(gate)
        fg, fu = (up * s).abs() * (1 + gate.abs() * (1 - s)), (gate * s).abs()
        n = torch.cat([fg, fu], 1) * ((H + 2) * mag[:M] + 16 * dh[:M].abs()).repeat(1, 2)
        check(dgu[:M], ref, n, -1, "dgu")
        assert torch.equal(dgu[M:].cpu(), d0[M:])


def test_swiglu_backward_formula_against_differences():
    """The derivative that the tests compare with, against central differences of the forward formula in 64 bits."""
    g = torch.Generator().manual_seed(3)
    gu, dh = torch.randn(5, 24, generator=g, dtype=torch.float64) * 2, torch.randn(5, 12, generator=g, dtype=torch.float64)
    f = lambda z: (dh * z[:, :12] * _sigmoid(z[:, :12]) * z[:, 12:]).sum()
    got = _swiglu_bwd(dh, gu, 12)
    step = 1e-5
    for i in range(5):
        for j in range(24):
            e = torch.zeros_like(gu)
            e[i, j] = step
            # third derivatives of silu are below 1: 1e-10 of |dh u|, and 1e-16 / 1e-5 of the sum's terms
            assert abs(float((f(gu + e) - f(gu - e)) / (2 * step) - got[i, j])) < 1e-8


# ------------------------------------------------------------------ combine, router

@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H,k", [(1, 8, 1), (3, 1000, 2), (129, 520, 7), (17, 2048, 16), (5, 16384, 3), (1100, 2048, 8)])
def test_combine_backward(T, H, k, dt):
    B = _B()
    g = torch.Generator().manual_seed(T + H)
    cap = T * k + 5
    inv = torch.randperm(cap, generator=g)[:T * k].to(torch.int32)
    inv[torch.rand(T * k, generator=g) < 0.3] = -1
    if T > 3:
        inv.view(T, k)[1] = -1                                # a token without a local expert
        inv[-1] = cap + 3                                     # outside the rows: no row
    dout, y, w = rnd(g, T, H, dt=dt), rnd(g, cap, H, dt=dt), rnd(g, T, k)
    d0 = rnd(g, cap, H, dt=dt)
    dy, dw = d0.cuda(), torch.full((T, k), 7.0, device="cuda")
    B.moe_combine_backward(dout.cuda(), y.cuda(), inv.cuda(), w.cuda(), dy, dw)
    ref, refw, magw = d0.double(), torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    touched = torch.zeros(cap, dtype=torch.bool)
    for p, pos in enumerate(inv.tolist()):
        if 0 <= pos < cap:
            t, j = divmod(p, k)
            ref[pos] = w[t, j].double() * dout[t].double()
            refw[t, j] = (dout[t].double() * y[pos].double()).sum()
            magw[t, j] = (dout[t].double() * y[pos].double()).abs().sum()
            touched[pos] = True
    check(dy[touched], ref[touched], ref[touched].abs(), 0, "dy_perm")
    assert torch.equal(dy.cpu()[~touched], d0[~touched])
    check(dw, refw, magw, H, "dtopk_w")
    assert (dw.cpu()[magw == 0] == 0).all()


def _gate(logits, ids, score, renorm, scale):
    """The weights of moe_route_topk at given ids, in 64 bits; ids outside the experts have weight 0."""
    E = logits.shape[1]
    ok = (ids >= 0) & (ids < E)
    p = torch.softmax(logits, 1) if score == "softmax" else _sigmoid(logits)
    w = torch.where(ok, p.gather(1, ids.clamp(0, E - 1)), torch.zeros((), dtype=torch.float64))
    if renorm:
        w = w / w.sum(1, keepdim=True)
    return w * scale


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(1, 1), (5, 5), (64, 6), (129, 8), (256, 16)])
def test_route_backward(E, k, renorm, score):
    B = _B()
    g = torch.Generator().manual_seed(E + k)
    for T in (1, 7, 130):
        logits = rnd(g, T, E, std=3.0)
        ids = torch.topk(logits + rnd(g, T, E), k, 1).indices.to(torch.int32)
        if T > 4:
            ids[1, 0], ids[2, -1] = -1, E                     # no such expert
            ids[3] = ids[3, 0]                                # the same expert in every slot
            logits[4, :] = -40.0
            logits[4, ids[4, 0]] = 40.0                       # scores at their ends
        # where every chosen slot is invalid a renormalised row has no weights: not made here
        if E == 1 and T > 4:
            ids[1, 0] = ids[2, -1] = 0
        dw = rnd(g, T, k)
        l = logits.double().requires_grad_(True)
        ref = torch.autograd.grad(_gate(l, ids.long(), score, renorm, 2.5), l, dw.double())[0]
        rp = B.route_params(E, k, score, renorm, routed_scale=2.5)
        for dt in (F32, BF):
            out = torch.full((T, E), 9.0, dtype=dt, device="cuda")
            B.moe_route_backward(logits.cuda(), ids.cuda(), dw.cuda(), rp, out)
            # every factor is at most 1 but the scale; terms: |d_j| + sum |d|, through exp (|l| + |lmax| < 60
            # roundings of its argument), sums over E and k
            mag = (2 * 2.5 * dw.double().abs().sum(1, keepdim=True)).expand(T, E)
            check(out, ref, mag, E + 2 * k + 60, f"dlogits {dt}")


def test_route_backward_rows_without_logits():
    B = _B()
    logits = torch.full((2, 8), -math.inf)
    logits[1, 3] = 0.5
    ids = torch.tensor([[0, 1], [3, 4]], dtype=torch.int32)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            out = torch.full((2, 8), 9.0, device="cuda")
            B.moe_route_backward(logits.cuda(), ids.cuda(), torch.ones(2, 2).cuda(), B.route_params(8, 2, score, renorm), out)
            assert torch.isfinite(out).all() and (out[0] == 0).all()


def test_route_backward_agrees_with_the_forward_routing():
    """Weights from moe_route_topk, their gradient against differences of moe_route_topk itself (fp32)."""
    B = _B()
    g = torch.Generator().manual_seed(11)
    T, H, E, k = 4, 128, 16, 3
    x, wr = rnd(g, T, H).cuda(), rnd(g, E, H, std=0.1).cuda()
    for score, renorm in (("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)):
        rp = B.route_params(E, k, score, renorm, routed_scale=1.5)
        ws = torch.empty(B.moe_route_workspace_size(T, H, E), dtype=torch.uint8, device="cuda")

        def route(bias, forced=None):
            ids, w, lg = (torch.empty(T, n, dtype=d, device="cuda") for n, d in ((k, torch.int32), (k, F32), (E, F32)))
            B.moe_route_topk(x, wr, rp, ids, w, ws, logits_out=lg, logit_bias=bias, forced_ids=forced)
            return ids, w, lg

        bias = torch.zeros(E, device="cuda")
        ids, w, lg = route(bias)
        dw = rnd(g, T, k).cuda()
        dl = torch.empty(T, E, device="cuda")
        B.moe_route_backward(lg, ids, dw, rp, dl)
        step = 2.0 ** -6
        for e in range(E):
            bias[e] = step
            up = route(bias, ids)[1]
            bias[e] = -step
            down = route(bias, ids)[1]
            bias[e] = 0.0
            diff = ((up.double() - down.double()) * dw.double()).sum(1) / (2 * step)
            # step^2 / 6 of third derivatives below 1.5 * 1 each, and 8 roundings of 2^-24 over 2 * step
            tol = dw.double().abs().sum(1) * 1.5 * (step ** 2 / 6 + 8 * 2.0 ** -24 / (2 * step))
            assert ((diff - dl[:, e].double()).abs() <= tol).all(), (score, renorm, e)


# ------------------------------------------------------------------ AdamW

HP = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, seed=77)


def _mix(x):
    x = np.uint32(x)
    with np.errstate(over="ignore"):
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0x7FEB352D)
        x = (x ^ (x >> np.uint32(15))) * np.uint32(0x846CA68B)
        return x ^ (x >> np.uint32(16))


def _random(n, q, t, seed):
    with np.errstate(over="ignore"):
        key = _mix(_mix(np.array([(seed + 0x9E3779B9 * t) % 2 ** 32], np.uint32)) + np.uint32(0x85EBCA77 * q % 2 ** 32))
        a = _mix(np.arange(n, dtype=np.uint32) ^ key)
        return a.astype(np.int64), _mix(a + np.uint32(0x9E3779B9)).astype(np.int64)


E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def _decode(codes, scale):
    c = codes.astype(np.int64)
    v = E4M3[np.minimum(c & 127, 126)] * np.where(c & 128, -1.0, 1.0)
    return v * np.repeat(2.0 ** (scale.astype(np.float64) - 127), 128)[:len(c)]


def _around(x, scale):
    """The two codes' values that |x| lies between (in the block's scale), in 64 bits."""
    s = np.repeat(2.0 ** (scale.astype(np.float64) - 127), 128)[:len(x)]
    y = np.abs(x) / s
    lo = np.searchsorted(E4M3, y, side="right") - 1
    return E4M3[lo] * s, E4M3[np.minimum(lo + 1, 126)] * s


@pytest.mark.parametrize("grad", [BF, F32], ids=["gbf16", "gf32"])
@pytest.mark.parametrize("param,master", [(F32, False), (BF, False), (BF, True)], ids=["f32", "bf16", "master"])
@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
def test_adamw(eight, param, master, grad):
    """Three steps of tensors of odd sizes: each against the formula in 64 bits from the state before it."""
    B = _B()
    sizes = [1, 7, 8, 127, 128, 129, 2048, 2049, 5000, 40000] + [3] * 60
    g = torch.Generator().manual_seed(1)
    p = [rnd(g, n, dt=param, std=0.5).cuda() for n in sizes]
    ma = [t.float() for t in p] if master else None
    if eight:
        m, v = ([torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda") for n in sizes] for _ in range(2))
        ms, vs = ([torch.zeros((n + 127) // 128, dtype=torch.uint8, device="cuda") for n in sizes] for _ in range(2))
    else:
        m, v = ([torch.zeros(n, device="cuda") for n in sizes] for _ in range(2))
        ms = vs = None
    gr = [torch.empty(n, dtype=grad, device="cuda") for n in sizes]
    table, hp = B.moe_adamw_table(p, gr, m, v, ms, vs, ma), B.adamw_params(**HP)
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    lr_scale, grad_scale = torch.tensor([0.5], device="cuda"), torch.tensor([0.25], device="cuda")
    lr = HP["lr"] * 0.5
    for t in (1, 2, 3):
        for i, x in enumerate(gr):
            x.copy_(rnd(g, sizes[i], std=10.0 ** (t - 2)))
            if t == 2:
                x[: sizes[i] // 2] = 0                        # states that only decay
        before = [[x.cpu().clone() for x in col] if col else None for col in (p, gr, m, v, ms, vs, ma)]
        step.add_(1)
        B.moe_adamw_step(table, hp, step, lr_scale=lr_scale, grad_scale=grad_scale)
        torch.cuda.synchronize()
        for i, n in enumerate(sizes):
            P, G, M, V, MS, VS, MA = (None if c is None else c[i] for c in before)
            gd = G.double().numpy() * 0.25
            if eight:
                m0 = _decode(M.view(torch.uint8).numpy(), MS.numpy())
                v0 = _decode(V.view(torch.uint8).numpy(), VS.numpy()) ** 2
            else:
                m0, v0 = M.double().numpy(), V.double().numpy()
            p0 = (MA if master else P).double().numpy()
            m1 = 0.9 * m0 + 0.1 * gd
            v1 = 0.95 * v0 + 0.05 * gd * gd
            den = np.sqrt(v1 / (1 - 0.95 ** t)) + 1e-8
            up = lr / (1 - 0.9 ** t) * m1 / den
            p1 = p0 * (1 - lr * 0.1) - up
            # fp32: 4 roundings in m and v (of their terms' magnitudes), 10 in the update, 3 in p
            u = 2.0 ** -24
            em = 4 * u * (0.9 * np.abs(m0) + 0.1 * np.abs(gd)) + 1e-44
            ev = 4 * u * v1 + 1e-44
            ep = 3 * u * np.abs(p0) + 12 * u * np.abs(up) + lr / (1 - 0.9 ** t) * em / den + 1e-44
            a, b = _random(n, i, t, HP["seed"])
            got = (ma if master else p)[i].double().cpu().numpy()
            if param == BF and not master:
                # floor(|p| / step + r / 2^16) steps, from a value off by at most ep
                def rounded(x):
                    s = 2.0 ** np.maximum(np.frexp(np.maximum(np.abs(x), 1e-300))[1] - 8, -133)
                    return np.sign(x) * np.floor(np.abs(x) / s + ((a & 0xFFF) * 16 + (b & 15)) / 65536) * s
                ok = (got == rounded(p1)) | ((got >= np.minimum(rounded(p1 - ep), rounded(p1 + ep))) &
                                             (got <= np.maximum(rounded(p1 - ep), rounded(p1 + ep))))
                assert ok.all(), (t, i, n)
            else:
                assert (np.abs(got - p1) <= ep + u * np.abs(p1)).all(), (t, i, n)
            if master:
                assert torch.equal(p[i], ma[i].to(BF)), "param is the master rounded"
            if not eight:
                assert (np.abs(m[i].double().cpu().numpy() - m1) <= em).all(), (t, i, n)
                assert (np.abs(v[i].double().cpu().numpy() - v1) <= ev).all(), (t, i, n)
                continue
            for x, codes, scale, r, root in ((m1, m[i], ms[i], a >> 12, False), (np.sqrt(v1), v[i], vs[i], b >> 12, True)):
                c, s = codes.view(torch.uint8).cpu().numpy(), scale.cpu().numpy()
                top = np.array([np.abs(x[j:j + 128]).max() for j in range(0, n, 128)])
                want = np.maximum(np.ceil(np.log2(np.maximum(top, 1e-300) / 448)), -127)
                near = np.abs(top / (448 * 2.0 ** want) - 1) < 1e-6                   # a maximum on a border
                near |= np.abs(top / (224 * 2.0 ** want) - 1) < 1e-6
                assert ((s.astype(int) - 127 == want) | near).all(), (t, i, n)
                val, (lo, hi) = np.abs(_decode(c, s)), _around(x, s)
                sc = np.repeat(2.0 ** (s.astype(np.float64) - 127), 128)[:n]
                frac = np.where(hi > lo, (np.abs(x) - lo) / np.where(hi > lo, hi - lo, 1), 0)
                # floor(x / code step + r / 2^20): up where the fraction passes 1 - r / 2^20; a tie of 1e-4 is open
                edge = frac + r / 2.0 ** 20 - 1
                exp_ = np.where(edge >= 0, hi, lo)
                if root:
                    exp_ = np.where((exp_ == 0) & (np.abs(x) > 0), 2.0 ** -9 * sc, exp_)
                ok = (val == exp_) | (np.abs(edge) < 1e-4) | (frac < 1e-4) | (frac > 1 - 1e-4)
                assert ok.all(), (t, i, n, "root" if root else "m", int((~ok).sum()))
                assert ((val >= lo) & (val <= hi) | ~(np.abs(edge) > 1e-4) | (frac < 1e-4) | (frac > 1 - 1e-4)).all()
                nz = np.abs(x) > 1e-30
                assert (np.sign(_decode(c, s))[nz & (val > 0)] == np.sign(x)[nz & (val > 0)]).all()
                if root:
                    assert ((c != 0) | (x == 0)).all(), "a nonzero second moment became 0"


def test_adamw_stochastic_rounding_is_unbiased():
    """A constant gradient far below half a bf16 step moves the mean of the weights as fp32 would."""
    B = _B()
    n = 1 << 16
    p = torch.ones(n, dtype=BF, device="cuda")
    gr = torch.ones(n, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    table = B.moe_adamw_table([p], [gr], [m], [v])
    hp = B.adamw_params(lr=2.0 ** -12, weight_decay=0.0, eps=1e-30, seed=5)
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    steps = 16
    for _ in range(steps):
        step.add_(1)
        B.moe_adamw_step(table, hp, step)
    # each step is -2^-12 exactly (m / sqrt(v) = 1 with bias correction).  Below 1 values are 2^-8 apart: one rounding
    # has variance at most 2^-16 / 4, so the mean of n elements over the steps has sigma <= 2^-9 sqrt(steps / n) = 3.1e-5.
    # Six sigma, and the update's own 1e-6.
    got = 1.0 - float(p.double().mean())
    assert abs(got - steps * 2.0 ** -12) < 6 * 2.0 ** -9 * math.sqrt(steps / n) + 1e-6, got


def test_adamw_graph_replays_follow_the_step():
    """A captured step replayed with a growing step count equals eager steps."""
    B = _B()
    n = 3001
    g = torch.Generator().manual_seed(2)

    def make():
        h = torch.Generator().manual_seed(4)
        p = rnd(h, n, dt=BF).cuda()
        m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
        ms, vs = (torch.zeros((n + 127) // 128, dtype=torch.uint8, device="cuda") for _ in range(2))
        gr = torch.zeros(n, device="cuda")
        return dict(p=p, m=m, v=v, ms=ms, vs=vs, g=gr, step=torch.zeros(1, dtype=torch.int32, device="cuda"),
                    table=B.moe_adamw_table([p], [gr], [m], [v], [ms], [vs]))

    hp = B.adamw_params(**HP)

    def one(s):
        s["step"].add_(1)
        B.moe_adamw_step(s["table"], hp, s["step"])

    a, b = make(), make()
    warm = make()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        one(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(b)
    for _ in range(5):
        grad = rnd(g, n).cuda()
        a["g"].copy_(grad)
        b["g"].copy_(grad)
        one(a)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("p", "m", "v", "ms", "vs", "step"):
            assert torch.equal(a[name], b[name]), name


# ------------------------------------------------------------------ the layer

def _layer_inputs(cid, dt, forced):
    import workloads as W
    cfg = W.get_config(cid, small=True).replace(wdt=dt, act=dt)
    inp = W.make_inputs(cfg, 3)
    if forced and inp["forced_ids"] is None:
        u = torch.rand(cfg.T, cfg.E, generator=torch.Generator().manual_seed(9))
        inp["forced_ids"] = torch.argsort(u, 1)[:, :cfg.k].to(torch.int32).contiguous()
    return cfg, inp


def _layer64(cfg, inp, weights, x, ids):
    """The layer in 64 bits at given expert ids; weights: dict of 64-bit tensors that may require gradients."""
    logits = x @ weights["w_router"][0].T
    if inp["logit_bias"] is not None:
        logits = logits + inp["logit_bias"].double()
    w = _gate(logits, ids, cfg.score, cfg.renormalize, cfg.routed_scale)
    out = torch.zeros_like(x)

    def swiglu(z, w13, w2):
        I = w2.shape[1]
        gu = z @ w13.T
        return (gu[:, :I] * _sigmoid(gu[:, :I]) * gu[:, I:]) @ w2.T

    for e in range(cfg.expert_begin, cfg.expert_end):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            y = swiglu(x[t], weights["w13"][e - cfg.expert_begin], weights["w2"][e - cfg.expert_begin])
            out = out.index_add(0, t, y * w[t, j, None])
    if "shared_w13" in weights:
        out = out + swiglu(x, weights["shared_w13"][0], weights["shared_w2"][0])
    return out


@pytest.mark.parametrize("cid,dt", [(1, "f32"), (2, "bf16"), (4, "bf16"), (5, "bf16")])
def test_train_layer_gradients(cid, dt):
    """Forward, backward twice (gradients add up), against 64-bit autograd of the whole layer at the same experts."""
    from combine_dual_overlap_amd import TrainLayer
    _B()
    cfg, inp = _layer_inputs(cid, dt, forced=False)
    layer = TrainLayer(inp)
    x = inp["x"].cuda()
    g = torch.Generator().manual_seed(8)
    dout = rnd(g, *inp["x"].shape, dt=inp["x"].dtype)
    print(f"train layer {cfg.name} {dt} T={cfg.T}", flush=True)
    out = layer.forward(x).clone()
    ids = layer.buf["ids"][:cfg.T].cpu().long()
    dx = layer.backward(dout.cuda()).clone()
    first = {n: t.clone() for n, t in layer.grads.items()}
    layer.forward(x)
    layer.backward(dout.cuda())
    torch.cuda.synchronize()
    w64 = {n: t.double().cpu().requires_grad_(True) for n, t in layer.weights.items()}
    x64 = inp["x"].double().requires_grad_(True)
    ref = _layer64(cfg, inp, w64, x64, ids)
    grads = torch.autograd.grad(ref, [x64, *w64.values()], dout.double())
    # bf16: x_perm exact; gu, h, y, dy, dgu, dx_perm, dlogits rounded once each, at most seven of them in one
    # chain, each off by 2^-8 at most and 2^-8 / sqrt(3) rms, with independent signs: sqrt(7) 2^-8 / sqrt(3) = 0.6 %.
    # fp32 sums of at most 6000 terms: 1e-4 with room.
    tol = 1e-2 if dt == "bf16" else 1e-4
    def rel(a, b):
        return float((a.double().cpu() - b).norm() / b.norm().clamp(min=1e-300))
    assert rel(out, ref.detach()) < tol
    for name, got, want in [("x", dx, grads[0])] + [(n, first[n], gr) for n, gr in zip(w64, grads[1:])]:
        r = rel(got, want)
        print(f"  d{name}: {r:.2e}")
        assert r < tol, (name, r)
    for n, t in layer.grads.items():
        # twice the same addend in fp32: exact
        assert torch.equal(t, 2 * first[n]), n


@pytest.mark.parametrize("states,master", [("f32", True), ("fp8", False)])
def test_train_layer_step_changes_the_forward(states, master):
    """One step moves every weight against its gradient's sign by about lr; the layer's own copies are updated."""
    from combine_dual_overlap_amd import TrainLayer
    _B()
    cfg, inp = _layer_inputs(2, "bf16", forced=True)
    layer = TrainLayer(inp, states=states, master=master, lr=2.0 ** -6, weight_decay=0.0, eps=1e-20)
    x = inp["x"].cuda()
    before = layer.forward(x).clone()
    g = torch.Generator().manual_seed(8)
    layer.backward(rnd(g, *x.shape, dt=BF).cuda())
    old = {n: t.clone() for n, t in layer.weights.items()}
    gr = {n: t.clone() for n, t in layer.grads.items()}
    layer.step()
    for n, t in layer.weights.items():
        d = (t.double() - old[n].double())
        has = gr[n].abs() > 1e-12
        # the first update is lr * sign(g); the weight is then rounded to bf16: off by a step, 2^-7 of the larger
        tol = 2.0 ** -6 * 1e-3 + 2.0 ** -7 * torch.maximum(t.abs().double(), old[n].abs().double())
        assert ((d + 2.0 ** -6 * torch.sign(gr[n].double())).abs() <= tol)[has].all(), n
        assert (d[gr[n] == 0] == 0).all(), n
    after = layer.forward(x)
    assert not torch.equal(before, after)
    with pytest.raises(RuntimeError):
        layer.step()


def test_train_layer_refuses_short_forced_ids():
    from combine_dual_overlap_amd import TrainLayer
    _B()
    cfg, inp = _layer_inputs(2, "bf16", forced=True)
    layer = TrainLayer(inp, T_max=2 * cfg.T)
    x = inp["x"].repeat(2, 1).cuda()
    with pytest.raises(ValueError):
        layer.forward(x)                                      # ids of half of these tokens
    with pytest.raises(RuntimeError):
        layer.backward(x)
    with pytest.raises(ValueError):
        layer.forward(torch.cat([x, x]))                      # more than T_max
    with pytest.raises(ValueError):
        layer.forward(x[:, :128].contiguous())


def test_train_layer_step_in_a_graph():
    """Forward, backward and step captured once and replayed three times equal three eager steps."""
    from combine_dual_overlap_amd import TrainLayer
    _B()
    cfg, inp = _layer_inputs(2, "bf16", forced=False)
    g = torch.Generator().manual_seed(8)
    kw = dict(states="fp8", master=False, lr=2.0 ** -8)
    x, dout = inp["x"].cuda(), rnd(g, *inp["x"].shape, dt=BF).cuda()
    a, b, warm = TrainLayer(inp, **kw), TrainLayer(inp, **kw), TrainLayer(inp, **kw)

    def one(layer):
        layer.forward(x)
        layer.backward(dout)
        layer.step()

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        one(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(b)
    for _ in range(3):
        x.copy_(rnd(g, *x.shape, dt=BF))
        one(a)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.buf["out"], b.buf["out"])
        for n in a.weights:
            assert torch.equal(a.weights[n], b.weights[n]), n
        for p, q in zip(a.m + a.v + a.m_scale + a.v_scale, b.m + b.v + b.m_scale + b.v_scale):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_train_layer_fewer_tokens_and_another_stream():
    """Calls of fewer tokens than T_max, and a whole step on another stream, equal a layer made for them."""
    from combine_dual_overlap_amd import TrainLayer
    _B()
    cfg, inp = _layer_inputs(2, "bf16", forced=False)
    x = inp["x"].cuda()
    g = torch.Generator().manual_seed(8)
    dout = rnd(g, *x.shape, dt=BF).cuda()
    a, b = TrainLayer(inp), TrainLayer(inp)
    a.forward(x)
    a.backward(dout)
    a.zero_grad()
    s = torch.cuda.Stream()
    for T in (37, 1):
        b = TrainLayer(inp, T_max=T)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            oa = a.forward(x[:T]).clone()
            da = a.backward(dout[:T]).clone()
        ob = b.forward(x[:T]).clone()
        db = b.backward(dout[:T]).clone()
        torch.cuda.synchronize()
        assert torch.equal(oa, ob) and torch.equal(da, db)
        for n in a.grads:
            assert torch.equal(a.grads[n], b.grads[n]), n
        a.zero_grad()


def test_train_layer_refuses_a_backward_without_its_forward():
    """After a step (the weights have moved) and after a forward pass that failed."""
    from combine_dual_overlap_amd import TrainLayer
    _B()
    cfg, inp = _layer_inputs(2, "bf16", forced=False)
    layer = TrainLayer(inp)
    x = inp["x"].cuda()
    layer.forward(x)
    layer.backward(x)
    layer.step()
    with pytest.raises(RuntimeError):
        layer.backward(x)
    layer.forward(x)
    with pytest.raises(ValueError):
        layer.forward(x.t().contiguous().t())                 # rows are not contiguous
    with pytest.raises(RuntimeError):
        layer.backward(x)


def test_adamw_table_holds_its_tensors():
    """The caller may drop its lists."""
    B = _B()
    p, g, m, v = ([torch.ones(256, device="cuda")] for _ in range(4))
    table = B.moe_adamw_table(p, g, m, v)
    kept = p[0]
    for t in (p, g, m, v):
        t.clear()
    assert [c[0].numel() for c in table.keep[:4]] == [256] * 4 and table.keep[0][0] is kept
    with pytest.raises(RuntimeError):
        B.moe_adamw_table([kept], [kept], [torch.zeros(256, device="cuda")], [torch.zeros(256, device="cuda")])


def test_adamw_large_tensor_equals_its_prefix():
    """Where a workgroup takes four groups of elements instead of one the results are the same, bit for bit: an
    element's random numbers depend on its place in the tensor only."""
    B = _B()
    n, cut = 17 * 1000 * 1000 + 5, 128 * 330
    g = torch.Generator(device="cuda").manual_seed(3)
    p = torch.randn(n, generator=g, device="cuda").to(BF)
    gr = torch.randn(n, generator=g, device="cuda").to(BF)
    codes = lambda k: torch.zeros(k, dtype=torch.uint8, device="cuda")

    def steps(p, gr):
        k = p.numel()
        st = [codes(k), codes(k), codes((k + 127) // 128), codes((k + 127) // 128)]
        table = B.moe_adamw_table([p], [gr], [st[0]], [st[1]], [st[2]], [st[3]])
        step = torch.zeros(1, dtype=torch.int32, device="cuda")
        for _ in range(2):
            step.add_(1)
            B.moe_adamw_step(table, B.adamw_params(lr=0.01, weight_decay=0.0), step)
        return st

    small = p[:cut].clone()
    old_tail = p[-1000:].clone()
    a, b = steps(p, gr), steps(small, gr[:cut].clone())
    assert torch.equal(p[:cut], small) and all(torch.equal(x[:y.numel()], y) for x, y in zip(a, b))
    # The last elements have moved against their gradients by 2 lr, but for: bf16's stochastic rounding, less than
    # 2^-10 twice for weights below 1/4; the second step's m and sqrt(v) from codes off by an eighth at most (where
    # |g| > 0.1 no code is denormal): m by 0.09 / 0.19 / 8 = 6 %, sqrt(v) by sqrt(1 + (1.125^2 - 1) / 2) - 1 = 6.5 %.
    d = (p[-1000:].float() - old_tail.float()) * torch.sign(gr[-1000:].float())
    near = (old_tail.abs().float() < 0.22) & (gr[-1000:].abs().float() > 0.1)
    assert (d[near] < -0.02 + 0.01 * 0.13 + 2.0 ** -9).all() and int(near.sum()) > 100
    big = gr[-1000:].abs().float() > 0.1
    assert (a[0][-1000:] != 0)[big].all() and (a[1][-1000:] != 0).all()


def test_adamw_more_tensors_than_a_launch_holds():
    """4100 tensors of three elements equal the same elements in one tensor (fp32 throughout: nothing is random)."""
    B = _B()
    n = 4100
    g = torch.Generator().manual_seed(5)
    flat = [rnd(g, n, 4).cuda() for _ in range(2)] + [torch.zeros(n, 4, device="cuda") for _ in range(2)]
    one = [t.clone().reshape(-1) for t in flat]
    rows = [[r[:3] for r in t] for t in flat]
    hp = B.adamw_params(lr=0.01)
    step = torch.ones(1, dtype=torch.int32, device="cuda")
    B.moe_adamw_step(B.moe_adamw_table(*rows), hp, step)
    before = flat[0][:, 3].clone()
    B.moe_adamw_step(B.moe_adamw_table(*([t] for t in one)), hp, step)
    for t, u in zip(flat, one):
        assert torch.equal(t[:, :3], u.view(n, 4)[:, :3])
    assert torch.equal(flat[0][:, 3], before) and (flat[2][:, 3] == 0).all()
