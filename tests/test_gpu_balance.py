"""The balanced gate and the balance loss on the GPU against their 64-bit forms."""
import math

import pytest
import torch

import block_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _B():
    from combine_dual_overlap_amd import binding
    return binding


def _select(logits, bias, k, load=True, **kw):
    B = _B()
    T, E = logits.shape
    rp = B.route_params(E, k, kw.get("score", "softmax"), kw.get("renormalize", False), kw.get("groups", 1),
                        kw.get("kept", 1), kw.get("topn", 1), kw.get("scale", 1.0))
    ids, w = torch.full((T, k), -7, dtype=torch.int32, device=DEV), torch.full((T, k), math.nan, device=DEV)
    n = torch.zeros(E, dtype=torch.int32, device=DEV) if load else None
    B.moe_route_select(logits.to(DEV), rp, ids, w, select_bias=None if bias is None else bias.to(DEV), load=n)
    return ids.cpu(), w.cpu(), None if n is None else n.cpu()


def _check_select(logits, bias, k, **kw):
    ids, w, load = _select(logits, bias, k, **kw)
    rid, rw, rload = O.select(logits, bias, k, kw.get("score", "softmax"), kw.get("renormalize", False),
                              kw.get("groups", 1), kw.get("kept", 1), kw.get("topn", 1), kw.get("scale", 1.0))
    assert torch.equal(ids, rid)
    # held in 64 bits, rounded once (the 64-bit errors are far below the 1 % that is added)
    assert ((w.double() - rw).abs() <= 1.01 * O.U * rw.abs() + 1e-45).all()
    assert torch.equal(load, rload)


CASES = [(1, 1, 1, {}), (1, 8, 8, {}), (3, 64, 6, {}), (5, 65, 1, dict(renormalize=True)), (4, 128, 8, dict(scale=2.5)),
         (130, 256, 16, {}), (33, 200, 8, dict(score="sigmoid", renormalize=True)),
         (67, 256, 8, dict(score="sigmoid", renormalize=True, groups=8, kept=4, topn=2, scale=2.5)),
         (9, 160, 6, dict(groups=8, kept=3, topn=1)), (9, 160, 6, dict(groups=32, kept=7, topn=4, score="sigmoid")),
         (5, 64, 1, dict(groups=64, kept=1, topn=1)), (5, 128, 16, dict(groups=64, kept=8, topn=2)),
         (7, 93, 5, dict(groups=3, kept=2, topn=3, renormalize=True)),
         # groups of 32, 16, 8 and 4 lanes, of 6, 12 and 3 lanes, of parts of lanes
         (9, 256, 8, dict(groups=2, kept=1, topn=4)), (9, 128, 8, dict(groups=4, kept=2, topn=3, score="sigmoid")),
         (601, 256, 8, dict(groups=16, kept=5, topn=4, score="sigmoid", renormalize=True)), (9, 64, 6, dict(groups=2, kept=1, topn=2)),
         (9, 192, 8, dict(groups=8, kept=4, topn=2)), (9, 60, 4, dict(groups=5, kept=2, topn=2)), (9, 180, 9, dict(groups=15, kept=4, topn=1)),
         (9, 252, 8, dict(groups=14, kept=5, topn=3, score="sigmoid"))]


@pytest.mark.parametrize("T,E,k,kw", CASES)
def test_select(T, E, k, kw):
    g = torch.Generator().manual_seed(T * 1000 + E)
    logits = torch.randn(T, E, generator=g) * 2
    bias = torch.randn(E, generator=g) * (0.05 if kw.get("score") == "sigmoid" else 0.3 / E)
    _check_select(logits, bias, k, **kw)
    _check_select(logits, None, k, **kw)


@pytest.mark.parametrize("kw", [{}, dict(score="sigmoid"), dict(groups=4, kept=2, topn=2),
                                dict(score="sigmoid", groups=4, kept=2, topn=2, renormalize=True)])
def test_select_ties_go_to_the_lower_index(kw):
    g = torch.Generator().manual_seed(4)
    logits = torch.randint(0, 3, (40, 96), generator=g).float()
    logits[0] = 0.0
    bias = torch.randint(0, 2, (96,), generator=g).float() * 0.125
    _check_select(logits, bias, 8, **kw)
    _check_select(logits, torch.zeros(96), 8, **kw)


@pytest.mark.parametrize("kw", [{}, dict(renormalize=True), dict(score="sigmoid", renormalize=True),
                                dict(groups=4, kept=2, topn=2), dict(score="sigmoid", groups=4, kept=1, topn=3)])
def test_select_masks(kw):
    """Rows without an expert, with fewer than k, with the lowest finite value, infinities and NaN."""
    inf, low = math.inf, torch.finfo(torch.float32).min
    g = torch.Generator().manual_seed(5)
    logits = torch.randn(12, 80, generator=g)
    logits[0] = -inf
    logits[1] = math.nan
    logits[2, 3:] = -inf
    logits[3] = low
    logits[4, 1:] = low
    logits[5, ::2] = -inf
    logits[6, 7] = inf
    logits[7, [5, 70]] = inf
    logits[8, 20:60] = math.nan
    logits[9] = inf
    logits[10, :79] = -inf
    _check_select(logits, torch.randn(80, generator=g) * 0.1, 5, **kw)
    _check_select(logits, None, 5, **kw)


def test_select_far_bias_and_near_scores():
    """Keys that fp32 would merge: scores one half step of fp32 apart at a bias of 1."""
    logits = torch.tensor([[0.0, 3e-8, 6e-8, -3e-8]]).repeat(3, 1) + torch.tensor([[0.0], [1.0], [-1.0]])
    _check_select(logits, torch.ones(4), 4, score="sigmoid")
    _check_select(torch.tensor([[1e-7, 0.0, 2e-7, 1e-7]]), torch.ones(4), 3)
    # scores that saturate in fp32 do not in 64 bits; a bias of one half decides against a full score
    _check_select(torch.tensor([[20.0, 25.0, 30.0, 18.0]]), torch.tensor([0.0, 0.0, -0.5, 0.5]), 4, score="sigmoid")


def test_select_adds_to_load_and_runs_without_it():
    logits = torch.randn(50, 16, generator=torch.Generator().manual_seed(6))
    B = _B()
    rp = B.route_params(16, 2)
    ids, w = torch.empty(50, 2, dtype=torch.int32, device=DEV), torch.empty(50, 2, device=DEV)
    load = torch.full((16,), 5, dtype=torch.int32, device=DEV)
    for _ in range(2):
        B.moe_route_select(logits.to(DEV), rp, ids, w, load=load)
    ref = O.select(logits, None, 2, "softmax")
    assert torch.equal(load.cpu(), 5 + 2 * ref[2])
    assert torch.equal(_select(logits, None, 2, load=False)[0], ref[0])
    empty = torch.empty(0, 16, device=DEV)
    B.moe_route_select(empty, rp, ids[:0], w[:0], load=load)
    assert torch.equal(load.cpu(), 5 + 2 * ref[2])


@pytest.mark.parametrize("dt,T,H,E,k,score", [(torch.bfloat16, 37, 256, 64, 6, "softmax"), (torch.float32, 5, 128, 8, 2, "sigmoid"),
                                              (torch.bfloat16, 1, 1024, 256, 8, "sigmoid")])
def test_balanced_route_is_the_selection_of_its_logits(dt, T, H, E, k, score):
    B = _B()
    g = torch.Generator().manual_seed(7)
    x, w = torch.randn(T, H, generator=g).to(dt), (torch.randn(E, H, generator=g) * H ** -0.5).to(dt)
    lb, sb = torch.randn(E, generator=g) * 0.3, torch.randn(E, generator=g) * 0.05
    rp = B.route_params(E, k, score, True)
    ids, tw = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    load, logits = torch.zeros(E, dtype=torch.int32, device=DEV), torch.empty(T, E, device=DEV)
    ws = torch.empty(max(256, B.moe_route_workspace_size(T, H, E)), dtype=torch.uint8, device=DEV)
    B.moe_route_balanced(x.to(DEV), w.to(DEV), rp, ids, tw, ws, select_bias=sb.to(DEV), load=load, logits_out=logits,
                         logit_bias=lb.to(DEV))
    l = logits.cpu()
    ref = x.double() @ w.double().t() + lb.double()
    # products summed in fp32: H half steps of the magnitudes' sum at most
    assert ((l.double() - ref).abs() <= H * O.U * (x.double().abs() @ w.double().abs().t() + lb.abs())).all()
    rid, rw, rload = O.select(l, sb, k, score, True)
    assert torch.equal(ids.cpu(), rid) and torch.equal(load.cpu(), rload)
    assert ((tw.cpu().double() - rw).abs() <= 1.01 * O.U * rw).all()


def test_bias_update():
    B = _B()
    for load in ([4, 4, 4, 4], [1, 2, 3, 10], [0, 0, 0, 0], [2 ** 31 - 1, 0, 1, 2 ** 31 - 1]):
        n = torch.tensor(load, dtype=torch.int32, device=DEV)
        bias = torch.tensor([0.5, -0.25, 0.0, 1.0], device=DEV)
        B.moe_route_bias_update(bias, n, 0.125)
        mean = sum(load) / 4
        want = [b + 0.125 * ((mean > v) - (mean < v)) for b, v in zip([0.5, -0.25, 0.0, 1.0], load)]
        assert bias.cpu().tolist() == want and n.cpu().tolist() == [0] * 4


@pytest.mark.parametrize("T,E,score,out,acc", [(1, 1, "softmax", "f32", False), (1, 256, "sigmoid", "f32", True),
                                               (7, 33, "softmax", "bf16", False), (300, 64, "softmax", "f32", True),
                                               (5000, 128, "sigmoid", "bf16", True), (4099, 200, "softmax", "f32", False)])
def test_balance_loss(T, E, score, out, acc):
    B = _B()
    dt = torch.float32 if out == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(T + E)
    logits = torch.randn(T, E, generator=g) * 2
    if T > 2:
        logits[1] = -math.inf
        logits[2, : E // 2] = -math.inf
        logits[0, 0] = math.nan
    load = torch.randint(0, 50, (E,), generator=g, dtype=torch.int32)
    load[0] += 1
    before = (torch.randn(T, E, generator=g) * 0.01 / T).to(dt)
    rp = B.route_params(E, 1, score)
    loss, d = torch.full((1,), math.nan, device=DEV), before.to(DEV)
    ws = torch.empty(B.moe_route_balance_loss_workspace_size(T, E), dtype=torch.uint8, device=DEV)
    B.moe_route_balance_loss(logits.to(DEV), load.to(DEV), rp, 0.25, loss, d, ws, accumulate=acc)
    rl, rd, bound = O.balance_loss(logits, load, 0.25, score)
    want = rd + before.double() if acc else rd
    assert ((d.cpu().double() - want).abs() <= bound + O.U * want.abs() + O.rounding(dt, want)).all()
    # every token's inner sum is fp32 (E terms), tokens are added in 64 bits
    assert abs(loss.item() - rl) <= 64 * O.U * abs(rl) + 0.25 * 64 * O.U


def test_balance_loss_without_load_or_tokens():
    B = _B()
    rp = B.route_params(8, 2)
    loss, d = torch.ones(1, device=DEV), torch.ones(4, 8, device=DEV)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    none = torch.zeros(8, dtype=torch.int32, device=DEV)
    B.moe_route_balance_loss(torch.randn(4, 8, device=DEV), none, rp, 1.0, loss, d, ws)
    assert loss.item() == 0 and d.abs().max().item() == 0
    loss.fill_(3)
    B.moe_route_balance_loss(torch.empty(0, 8, device=DEV), none, rp, 1.0, loss, torch.empty(0, 8, device=DEV), ws)
    assert loss.item() == 0


def test_gate_captured_and_on_a_stream():
    """The whole gate of a training step, captured and replayed with new inputs in place."""
    B = _B()
    T, E, k = 70, 64, 4
    rp = B.route_params(E, k, "sigmoid", True)
    logits, bias = torch.empty(T, E, device=DEV), torch.zeros(E, device=DEV)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    load, loss, d = torch.zeros(E, dtype=torch.int32, device=DEV), torch.empty(1, device=DEV), torch.empty(T, E, device=DEV)
    ws = torch.empty(B.moe_route_balance_loss_workspace_size(T, E), dtype=torch.uint8, device=DEV)

    def step():
        B.moe_route_select(logits, rp, ids, w, select_bias=bias, load=load)
        B.moe_route_balance_loss(logits, load, rp, 0.1, loss, d, ws)
        B.moe_route_bias_update(bias, load, 0.01)

    logits.normal_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    bias.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ref_bias = torch.zeros(E)
    for i in range(3):
        l = torch.randn(T, E, generator=torch.Generator().manual_seed(i))
        logits.copy_(l)
        graph.replay()
        torch.cuda.synchronize()
        rid, rw, rload = O.select(l, ref_bias, k, "sigmoid", True)
        rl, rd, bound = O.balance_loss(l, rload, 0.1, "sigmoid")
        assert torch.equal(ids.cpu(), rid) and abs(loss.item() - rl) <= 64 * O.U * (abs(rl) + 0.1)
        assert ((d.cpu().double() - rd).abs() <= bound + 2 * O.U * rd.abs()).all()
        ref_bias = (ref_bias + 0.01 * torch.sign(rload.float().mean() - rload.float())).float()
        assert torch.equal(bias.cpu(), ref_bias) and load.abs().sum().item() == 0
