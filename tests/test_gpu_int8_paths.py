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
