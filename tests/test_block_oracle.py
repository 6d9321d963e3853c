"""The 64-bit forms of block_oracle against differences and against each other (CPU)."""
import math

import pytest
import torch

import block_oracle as O


def _diff(f, x, step=1e-6):
    """Central differences of a scalar function at x (float64)."""
    g = torch.zeros_like(x)
    flat, gf = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        old = flat[i].item()
        flat[i] = old + step
        hi = f(x)
        flat[i] = old - step
        lo = f(x)
        flat[i] = old
        gf[i] = (hi - lo) / (2 * step)
    return g


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_loss_gradient_is_its_difference(score):
    torch.manual_seed(1)
    l = torch.randn(5, 7, dtype=torch.float64)
    load = torch.tensor([3, 0, 4, 1, 1, 5, 1], dtype=torch.int32)
    _, d, _ = O.balance_loss(l, load, 0.3, score)
    num = _diff(lambda x: O.balance_loss(x, load, 0.3, score)[0], l.clone())
    assert (d - num).abs().max() < 1e-9


@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post", [True, False])
def test_norm_gradients_are_their_differences(kind, post):
    torch.manual_seed(2)
    T, H, eps = 3, 8, 1e-3
    y, d = torch.randn(T, H, dtype=torch.float64), torch.randn(T, H, dtype=torch.float64)
    w = torch.rand(H, dtype=torch.float64) + 0.5 if post else None
    gate = {"none": None, "channel": torch.randn(H), "token": torch.rand(T, 1), "full": torch.randn(T, H)}[kind]
    gate = None if gate is None else gate.double()

    def loss(y, w, gate):
        return float((d * O.block_out(y, y.abs(), None, eps, w, gate, 0.7)["out"]).sum())

    rstd = 1 / torch.sqrt((y * y).mean(1) + eps)
    got = O.norm_backward(d, y, rstd, w, gate, kind, 0.7, None)
    assert (got["dy"][0] - _diff(lambda v: loss(v, w, gate), y.clone())).abs().max() < 1e-8
    if post:
        assert (got["dw"][0] - _diff(lambda v: loss(y, v, gate), w.clone())).abs().max() < 1e-8
    if gate is not None:
        assert (got["dgate"][0] - _diff(lambda v: loss(y, w, v), gate.clone())).abs().max() < 1e-8


def test_select_without_bias_is_top_k_of_the_scores():
    torch.manual_seed(3)
    l = torch.randn(9, 12)
    ids, w, load = O.select(l, None, 3, "softmax")
    top = torch.topk(torch.softmax(l.double(), 1), 3)
    assert torch.equal(ids.long(), top.indices) and (w - top.values).abs().max() < 1e-15
    assert torch.equal(load, torch.bincount(ids.flatten(), minlength=12).int())
    # groups: only experts of the best group are chosen
    ids, _, _ = O.select(l, None, 3, "sigmoid", groups=3, kept=1, topn=2)
    best = torch.topk(torch.sigmoid(l.double()).view(9, 3, 4), 2, dim=2).values.sum(2).argmax(1)
    assert torch.equal(ids.long() // 4, best[:, None].expand(9, 3))


def test_select_masks():
    inf = math.inf
    l = torch.tensor([[-inf] * 4, [0.0, -inf, math.nan, -inf], [1.0, inf, 0.0, inf]])
    ids, w, load = O.select(l, torch.tensor([0.0, 5.0, 0.0, 0.0]), 2, "softmax")
    assert ids.tolist() == [[0, 1], [0, 1], [1, 3]]
    assert w.tolist() == [[0, 0], [1, 0], [0.5, 0.5]] and load.tolist() == [1, 1, 0, 1]


def test_quantize_rounds_to_nearest_even_and_marks_what_is_not_finite():
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5, -126.5], [0.0] * 5, [1.0, math.inf, 0, 0, 0], [math.nan, 1, 2, 3, 4]])
    q, s = O.quantize(x)
    # 127 * fp32(1 / 127) = 1 exactly: the halves are ties
    assert s[0] == 1.0 and q[0].tolist() == [127, 0, 2, -2, -126] and s[1] == 0 and q[1:].abs().sum() == 0
    assert torch.isnan(s[2:]).all()
