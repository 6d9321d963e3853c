"""Integer products where a workgroup walks several tiles, and the SwiGLU of integer experts to fp32's last places."""
import pytest
import torch

import block_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _B():
    from combine_dual_overlap_amd import binding
    return binding


def _int8(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)


@pytest.mark.parametrize("rows,N", [(1, 64), (40, 64), (300, 512)])
def test_swiglu_is_rounded_like_fp32_arithmetic(rows, N):
    """h of gates between -100 and 100 against silu in 64 bits of the same fp32 gate and up values."""
    B = _B()
    g = torch.Generator().manual_seed(rows)
    K = 256
    a, b = _int8(g, rows, K), _int8(g, 1, 2 * N, K)
    s, t = 1e-5 * (1 + torch.rand(rows, generator=g)), 10.0 * (1 + torch.rand(1, 2 * N, generator=g))
    h = torch.full((rows, N), 9.0, device=DEV)
    B.moe_grouped_swiglu_int8(a.to(DEV), s.to(DEV), b.to(DEV), t.to(DEV), None, h)
    gate, up = O.int8_product(a, s, b[0], t[0]).chunk(2, dim=1)
    assert rows < 40 or (gate.min() < -60 and gate.max() > 60)
    want = gate.double() * torch.sigmoid(gate.double()) * up.double()
    # half steps: the exponential 2 (a unit in the last place), 1 + e 1, the quotient 1, the product with u 1, and a fiftieth
    # for their products.  (Below -87 the quotient is of a number above 2^126, and may be off by all that is left of it.)
    bound = 5.1 * O.U * want.abs() + (gate * up).abs().double() * 2.0 ** -126 + 2.0 ** -126
    assert ((h.cpu().double() - want).abs() <= bound).all()


@pytest.mark.filterwarnings("ignore:.*encountered:RuntimeWarning")      # (infinities, on purpose)
def test_swiglu_of_gates_that_overflow():
    """Gates that are infinite, NaN or at fp32's ends: what g / (1 + exp(-g)) * u is in fp32."""
    B = _B()
    g = torch.Generator().manual_seed(3)
    rows, K, N = 40, 64, 32
    a, b = _int8(g, rows, K), _int8(g, 1, 2 * N, K)
    s, t = torch.full((rows,), 1e-3), torch.full((1, 2 * N), 1e-2)
    s[1::5], s[2::5], s[3::5] = 1e36, torch.inf, torch.nan
    t[0, :N:3] = 1e36
    t[0, 1:N:3] = 10.0
    h = torch.full((rows, N), 9.0, device=DEV)
    B.moe_grouped_swiglu_int8(a.to(DEV), s.to(DEV), b.to(DEV), t.to(DEV), None, h)
    gate, up = O.int8_product(a, s, b[0], t[0]).chunk(2, dim=1)
    assert (gate == torch.inf).any() and (gate == -torch.inf).any() and gate.isnan().any()
    want, got = gate / (1.0 + torch.exp(-gate)) * up, h.cpu()
    # (between -87 and -88.8 the quotient is 0 where it is below 2^-126, and up may be infinite)
    near = (gate > -87.0) | (gate < -88.8) | gate.isnan()
    assert torch.equal(got.isnan()[near], want.isnan()[near])
    wild = near & want.isinf()
    assert torch.equal(got[wild], want[wild])
    fine = near & want.isfinite()
    # two such calculations of at most 5.1 half steps each
    assert ((got[fine].double() - want[fine].double()).abs() <= 10.2 * O.U * want[fine].abs().double() + 2.0 ** -126).all()


def _ragged(g, experts, mean):
    """Rows of each expert around `mean`, every ninth without any."""
    n = torch.randint(max(1, mean // 2), mean + mean // 2 + 1, (experts,), generator=g)
    n[4::9] = 0
    return n.tolist()


# 64 experts of about 24 rows are tiles of 32 x 128 (512 workgroups, three stages in flight), 48 of about 90 rows tiles of
# 128 x 128 (512 workgroups, two stages); with 2048 columns there are more tiles than workgroups.  A tile is one stage, two
# with a short one, and four.
WALKS = [(64, 24, 2048), (64, 24, 2056), (48, 90, 2048), (48, 90, 2184)]
STAGES = [16, 128, 144, 400]


@pytest.mark.parametrize("K", STAGES)
@pytest.mark.parametrize("experts,mean,N", WALKS)
def test_products_of_many_tiles(experts, mean, N, K):
    """Bit for bit: whole sums, then an fp32 rounding for each scale, then one to the result's type."""
    B = _B()
    g = torch.Generator().manual_seed(experts + N + K)
    n = _ragged(g, experts, mean)
    M = sum(n)
    high = 32 if mean <= 32 else 128
    assert sum(-(-r // high) for r in n) * -(-N // 128) > 640
    cap = M + 5
    a, b = _int8(g, cap, K), _int8(g, experts, N, K)
    s, t = 0.01 * (1 + torch.rand(cap, generator=g)), 0.01 * (1 + torch.rand(experts, N, generator=g))
    off = torch.tensor([sum(n[:e]) for e in range(experts + 1)], dtype=torch.int32)
    want = torch.full((cap, N), 9.0)
    for e in range(experts):
        i, j = int(off[e]), int(off[e + 1])
        if j > i:
            want[i:j] = O.int8_product(a[i:j], s[i:j], b[e], t[e])
    dev = [v.to(DEV) for v in (a, s, b, t, off)]
    for dt in (torch.float32, torch.bfloat16):
        for _ in range(3):
            c = torch.full((cap, N), 9.0, dtype=dt, device=DEV)
            B.moe_grouped_gemm_int8(*dev, c)
            assert torch.equal(c.cpu(), want.to(dt)), dt


@pytest.mark.parametrize("K", STAGES)
@pytest.mark.parametrize("experts,mean,I", [(64, 24, 1032), (48, 90, 1024)])
def test_swiglu_of_many_tiles(experts, mean, I, K):
    B = _B()
    g = torch.Generator().manual_seed(experts + I + K)
    n = _ragged(g, experts, mean)
    cap = sum(n) + 5
    a, b = _int8(g, cap, K), _int8(g, experts, 2 * I, K)
    s, t = 1e-3 * (1 + torch.rand(cap, generator=g)), 0.01 * (1 + torch.rand(experts, 2 * I, generator=g))
    off = torch.tensor([sum(n[:e]) for e in range(experts + 1)], dtype=torch.int32)
    want, bound = torch.full((cap, I), 9.0, dtype=torch.float64), torch.zeros(cap, I, dtype=torch.float64)
    for e in range(experts):
        i, j = int(off[e]), int(off[e + 1])
        if j > i:
            gate, up = O.int8_product(a[i:j], s[i:j], b[e], t[e]).double().chunk(2, dim=1)
            want[i:j] = gate * torch.sigmoid(gate) * up
            bound[i:j] = 5.1 * O.U * want[i:j].abs() + 2.0 ** -126 * (1 + (gate * up).abs())      # as above
    dev = [v.to(DEV) for v in (a, s, b, t, off)]
    for dt in (torch.float32, torch.bfloat16):
        h = torch.full((cap, I), 9.0, dtype=dt, device=DEV)
        B.moe_grouped_swiglu_int8(*dev, h)
        far = (h.cpu().double() - want).abs()
        assert (far <= bound + (O.rounding(dt, want.abs() + bound) if dt == torch.bfloat16 else 0.0)).all(), dt
