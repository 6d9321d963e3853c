"""Products of 8-bit integers on the GPU: exact sums, so most results are compared bit for bit."""
import math

import pytest
import torch

import block_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _B():
    from combine_dual_overlap_amd import binding
    return binding


def _rand_int8(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)


def _offsets(counts):
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int32), off


# ------------------------------------------------------------------ quantisation

@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,K", [(1, 16), (3, 48), (5, 512), (4, 528), (2, 2048), (3000, 1024), (2, 7168), (3, 16384), (1, 65552)])
def test_quant_rows(n, K, dt):
    B = _B()
    g = torch.Generator().manual_seed(n + K)
    x = (torch.randn(n, K, generator=g) * 2.0 ** torch.randint(-20, 20, (n, 1), generator=g)).to(dt)
    if n > 2:
        x[0] = 0
        x[1] = torch.randint(-127, 128, (K,), generator=g).to(dt) / 2      # ties where the largest is 63.5
        x[1, 0] = 63.5
        x[2] = (torch.randn(K, generator=g) * 1e-40).to(dt)                # subnormal scales
    q, s = torch.full((n, K), 99, dtype=torch.int8, device=DEV), torch.empty(n, device=DEV)
    B.moe_quant_int8_rows(x.to(DEV), q, s)
    rq, rs = O.quantize(x)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu(), rq)


def test_quant_rows_extremes():
    B = _B()
    big, tiny, sub = torch.finfo(torch.float32).max, torch.finfo(torch.float32).tiny, 2.0 ** -149
    x = torch.zeros(9, 16)
    x[0, :3] = torch.tensor([big, -big, big / 254])
    x[1, :3] = torch.tensor([tiny, -tiny / 2, tiny / 254])
    x[2, :3] = torch.tensor([sub, -sub, 0])
    x[3, :3] = torch.tensor([100 * sub, -50 * sub, sub])
    x[4, :3] = torch.tensor([190 * sub, -190 * sub, 95 * sub])
    x[5, 2] = math.inf
    x[6, 3] = math.nan
    x[7, :2] = torch.tensor([-math.inf, math.nan])
    x[8, 5] = -0.0
    q, s = torch.empty(9, 16, dtype=torch.int8, device=DEV), torch.empty(9, device=DEV)
    B.moe_quant_int8_rows(x.to(DEV), q, s)
    rq, rs = O.quantize(x)
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu().nan_to_num(-1), rs.nan_to_num(-1))
    # rows of more than two axes
    w = torch.randn(3, 5, 32, device=DEV)
    q, s = torch.empty(3, 5, 32, dtype=torch.int8, device=DEV), torch.empty(3, 5, device=DEV)
    B.moe_quant_int8_rows(w, q, s)
    rq, rs = O.quantize(w.cpu().view(15, 32))
    assert torch.equal(q.cpu().view(15, 32), rq) and torch.equal(s.cpu().view(15), rs)
    B.moe_quant_int8_rows(w[:0], q[:0], s[:0])


# ------------------------------------------------------------------ dispatch

@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H,k,E,lo,hi", [(1, 16, 1, 1, 0, 1), (37, 272, 3, 8, 0, 8), (700, 128, 8, 64, 16, 48), (5000, 64, 2, 16, 0, 16),
                                           (64, 7168, 4, 32, 3, 4)])
def test_dispatch(T, H, k, E, lo, hi, dt):
    B = _B()
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(dt)
    ids = torch.argsort(torch.rand(T, E, generator=g), dim=1)[:, :k].to(torch.int32).contiguous()
    n, E_loc = T * k, hi - lo
    i32 = lambda m: torch.full((m,), -9, dtype=torch.int32, device=DEV)
    cnt, off, perm, inv = i32(E_loc), i32(E_loc + 1), i32(n), i32(n)
    ws = torch.empty(max(256, B.moe_dispatch_workspace_size(T, k, E_loc)), dtype=torch.uint8, device=DEV)
    plain = torch.zeros(n, H, dtype=dt, device=DEV)
    B.moe_dispatch(x.to(DEV), ids.to(DEV), E, lo, hi, cnt, off, perm, inv, plain, ws)
    want = [t.clone() for t in (cnt, off, perm, inv)]
    for t in (cnt, off, perm, inv):
        t.fill_(-9)
    xq, xs = torch.full((n, H), 77, dtype=torch.int8, device=DEV), torch.full((n,), -5.0, device=DEV)
    B.moe_dispatch_int8(x.to(DEV), ids.to(DEV), E, lo, hi, cnt, off, perm, inv, xq, xs, ws)
    M = int(off[-1])
    for a, b in zip((cnt, off, inv), (want[0], want[1], want[3])):
        assert torch.equal(a, b)
    assert torch.equal(perm[:M], want[2][:M])
    rq, rs = O.quantize(plain[:M].cpu()) if M else (xq[:0].cpu(), xs[:0].cpu())
    assert torch.equal(xq[:M].cpu(), rq) and torch.equal(xs[:M].cpu(), rs)
    assert (xq[M:] == 77).all() and (xs[M:] == -5).all()          # rows behind the last are left as they were


# ------------------------------------------------------------------ products

PRODUCTS = [([1], 8, 16), ([5], 24, 48), ([0, 3, 0], 128, 128), ([31, 1, 33], 136, 272), ([64, 0, 65, 200], 264, 144),
            ([129, 300], 512, 256), ([1000], 72, 2048), ([700, 300, 257], 1024, 400), ([2], 2816, 2048),
            ([260] * 40, 520, 128), ([3000], 2048, 64), ([128, 5, 0, 77], 384, 16),
            # tiles of 32 x 128 with few rows, 128 x 128 and 256 x 256 with ragged ones
            ([1, 2] * 12, 1032, 272), ([0, 1, 31, 32, 33, 64, 5] + [2] * 8, 1416, 400), ([17] * 30, 520, 1040),
            ([1] * 64, 264, 16), ([129, 500, 1, 127, 260], 4104, 80), ([600, 333, 511, 257, 513], 8200, 272),
            ([513, 0, 1, 900], 12296, 64)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,N,K", PRODUCTS)
def test_product(counts, N, K, out):
    B = _B()
    g = torch.Generator().manual_seed(sum(counts) + N + K)
    E, (offsets, off) = len(counts), _offsets(counts)
    cap = off[-1] + 3
    a, b = _rand_int8(g, cap, K), _rand_int8(g, E, N, K)
    asc, bsc = torch.rand(cap, generator=g) * 0.1, torch.rand(E, N, generator=g) * 0.01
    bsc[0, 0] = 0.0
    c = torch.full((cap, N), 7.0, dtype=out, device=DEV)
    B.moe_grouped_gemm_int8(a.to(DEV), asc.to(DEV), b.to(DEV), bsc.to(DEV), offsets.to(DEV), c)
    got = c.cpu()
    for e in range(E):
        r = slice(off[e], off[e + 1])
        assert torch.equal(got[r], O.int8_product(a[r], asc[r], b[e], bsc[e]).to(out)), e
    assert (got[off[-1]:] == 7).all()
    if E == 1:
        c.fill_(7)
        B.moe_grouped_gemm_int8(a.to(DEV), asc.to(DEV), b.to(DEV), bsc.to(DEV), None, c)
        assert torch.equal(c.cpu(), O.int8_product(a, asc, b[0], bsc[0]).to(out))


def test_product_extremes():
    """The largest sums, and scales that are not finite."""
    B = _B()
    K = 1 << 17
    a, b = torch.full((2, K), 127, dtype=torch.int8), torch.full((1, 8, K), 127, dtype=torch.int8)
    b[0, 1] = -127
    asc, bsc = torch.tensor([1.0, math.nan]), torch.ones(1, 8)
    bsc[0, 3] = math.inf
    c = torch.empty(2, 8, device=DEV)
    B.moe_grouped_gemm_int8(a.to(DEV), asc.to(DEV), b.to(DEV), bsc.to(DEV), None, c)
    want = O.int8_product(a, asc, b[0], bsc[0])
    assert torch.equal(c.cpu()[0], want[0]) and torch.isnan(c[1]).all()
    # offsets that point outside of the rows are cut off
    a, b = torch.ones(6, 16, dtype=torch.int8, device=DEV), torch.ones(2, 8, 16, dtype=torch.int8, device=DEV)
    c = torch.zeros(6, 8, device=DEV)
    B.moe_grouped_gemm_int8(a, torch.ones(6, device=DEV), b, torch.ones(2, 8, device=DEV),
                            torch.tensor([-3, 2, 99], dtype=torch.int32, device=DEV), c)
    assert (c == 16).all()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,I,H", [([1], 8, 16), ([0, 40, 3], 72, 48), ([33, 130], 136, 256), ([600, 300], 264, 128), ([300] * 9, 1032, 64),
                                        ([1, 0, 17, 16] * 6, 392, 208), ([33, 300, 1] * 2, 2056, 144), ([600, 333, 511, 257, 513], 4104, 272)])
def test_swiglu(counts, I, H, out):
    B = _B()
    g = torch.Generator().manual_seed(sum(counts) + I)
    E, (offsets, off) = len(counts), _offsets(counts)
    x, w = _rand_int8(g, off[-1] + 2, H), _rand_int8(g, E, 2 * I, H)
    xs, ws = torch.rand(off[-1] + 2, generator=g) * 0.02, torch.rand(E, 2 * I, generator=g) * 0.02
    xs[0] = 0.5                                       # pre-activations of some hundred
    h = torch.full((off[-1] + 2, I), 3.0, dtype=out, device=DEV)
    B.moe_grouped_swiglu_int8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), offsets.to(DEV), h)
    got = h.cpu()
    for e in range(E):
        r = slice(off[e], off[e + 1])
        want, bound = O.swiglu_int8(x[r], xs[r], w[e], ws[e])
        assert ((got[r].double() - want).abs() <= bound + O.rounding(out, want)).all()
    assert (got[off[-1]:] == 3).all()


@pytest.mark.parametrize("counts,H,I", [([1], 16, 16), ([3, 0, 50], 64, 48), ([130, 0, 257, 1], 256, 208), ([700], 144, 512),
                                        ([280] * 10, 512, 96), ([1, 2, 0, 3] * 10, 528, 272), ([1, 1], 16, 8208)])
def test_ffn(counts, H, I):
    B = _B()
    g = torch.Generator().manual_seed(sum(counts) + H)
    E, (offsets, off) = len(counts), _offsets(counts)
    cap = off[-1] + 5
    x = torch.randn(cap, H, generator=g)
    xq, xs = O.quantize(x)
    w13, s13 = O.quantize(torch.randn(E * 2 * I, H, generator=g) * H ** -0.5)
    w2, s2 = O.quantize(torch.randn(E * H, I, generator=g) * I ** -0.5)
    w13, s13, w2, s2 = w13.view(E, 2 * I, H), s13.view(E, 2 * I), w2.view(E, H, I), s2.view(E, H)
    xs[off[-1] - 1] = math.nan                       # a row that was not finite
    y = torch.full((cap, H), 5.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(B.moe_ffn_int8_workspace_size(cap, I), dtype=torch.uint8, device=DEV)
    args = [t.to(DEV) for t in (xq, xs, offsets, w13, s13, w2, s2)]
    B.moe_grouped_ffn_int8(*args, y, ws)
    got = y.cpu()
    for e in range(E):
        r = slice(off[e], off[e + 1])
        fine = torch.isfinite(xs[r])
        if not fine.any():
            continue
        want, bound = O.ffn_int8(xq[r][fine], xs[r][fine], w13[e], s13[e], w2[e], s2[e])
        assert ((got[r][fine].double() - want).abs() <= bound + O.rounding(torch.bfloat16, want)).all()
    assert torch.isnan(got[off[-1] - 1]).all() and (got[off[-1]:] == 5).all()
    # captured and replayed, the workspace full of something else in between
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_grouped_ffn_int8(*args, y, ws)
    for _ in range(3):
        y.fill_(5)
        ws.random_(0, 255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu().nan_to_num(-1), got.nan_to_num(-1))


def test_offsets_past_32_bits():
    """Rows whose byte offsets (and elements of c) pass 2^32."""
    B = _B()
    rows, N, K = 140000, 32768, 16
    a = torch.ones(rows, K, dtype=torch.int8, device=DEV)
    a[-3:] = torch.tensor([[2], [-3], [5]], dtype=torch.int8, device=DEV)
    b = torch.ones(1, N, K, dtype=torch.int8, device=DEV)
    c = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)
    B.moe_grouped_gemm_int8(a, torch.ones(rows, device=DEV), b, torch.ones(1, N, device=DEV), None, c)
    assert (c[:-3:997] == 16).all() and c[-3:, ::1001].float().unique(dim=1).flatten().tolist() == [32, -48, 80]
    q, s = torch.empty(rows, N, dtype=torch.int8, device=DEV), torch.empty(rows, device=DEV)
    B.moe_quant_int8_rows(c, q, s)
    assert (q[:-3:997] == 127).all() and q[-3:, ::1001].float().unique(dim=1).flatten().tolist() == [127, -127, 127]
    assert s[-1].item() == 80 * float(O.INV127)
