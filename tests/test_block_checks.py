"""Settings and buffers that the layers, the balanced gate and the build refuse or put right, without a GPU."""
import ctypes

import pytest
import torch

A = 1 << 20       # aligned made-up address


def test_train_layer_refuses_rates_that_its_steps_refuse():
    """An infinite bias_rate was refused by step() only, after the weights had moved."""
    import workloads as W
    from combine_dual_overlap_amd import TrainLayer
    inp = W.make_inputs(W.get_config(1, small=True))
    inp["forced_ids"] = None
    for bad in (float("inf"), float("nan"), -0.5, 3.41e38):
        for name in ("bias_rate", "balance_coef"):
            with pytest.raises(ValueError, match="balance_coef and bias_rate"):
                TrainLayer(inp, device="cpu", **{name: bad})


def test_integer_weights_come_with_a_scale_per_row():
    """int8 weights were run with whatever scales stood beside them: shorter ones were read behind their end."""
    import workloads as W
    from combine_dual_overlap_amd import DeviceLayer
    cfg = W.get_config(2, small=True)
    inp = W.make_inputs(cfg)
    E, H, I = cfg.E, cfg.H, cfg.I
    good = dict(w13=torch.zeros(E, 2 * I, H, dtype=torch.int8), w2=torch.zeros(E, H, I, dtype=torch.int8),
                w13_scale=torch.ones(E, 2 * I), w2_scale=torch.ones(E, H))
    with pytest.raises(ValueError, match="device tensor"):           # nothing wrong but the device
        DeviceLayer({**inp, **good}, device="cpu")
    more = dict(good, w13=torch.zeros(E + 1, 2 * I, H, dtype=torch.int8), w13_scale=torch.ones(E + 1, 2 * I))
    with pytest.raises(ValueError, match="device tensor"):           # (experts behind the last are not used)
        DeviceLayer({**inp, **more}, device="cpu")
    for name, bad in (("w13", torch.ones(E, 2 * I // 128, H // 128)), ("w2", torch.ones(E, 1)), ("w2", torch.ones(E, H).double()),
                      ("w13", None), ("w2", torch.ones(E - 1, H))):
        with pytest.raises(ValueError, match=f"{name}: int8"):
            DeviceLayer({**inp, **good, name + "_scale": bad}, device="cpu")
    for name, bad in (("w2", inp["w2"]), ("w13", good["w13"][:, :-16]), ("w2", good["w2"][:-1])):
        with pytest.raises(ValueError, match=f"{name}: int8"):
            DeviceLayer({**inp, **good, name: bad}, device="cpu")


def test_gate_refuses_buffers_that_stand_for_two():
    from combine_dual_overlap_amd import binding as B
    L = B.lib()
    p = B.route_params(64, 6)
    bad = B.MOE_ERR_INVALID_ARG

    def select(l=A, b=2 * A, ids=3 * A, w=4 * A, load=5 * A):
        return L.moe_route_select(l, 8, b, ctypes.byref(p), ids, w, load, None)

    for kw in (dict(load=4 * A), dict(load=2 * A), dict(b=4 * A), dict(b=3 * A)):
        assert select(**kw) == bad, kw

    need = B.moe_route_workspace_size(8, 256, 64)

    def balanced(**kw):
        a = dict(x=A, wr=2 * A, lb=3 * A, sb=4 * A, lo=5 * A, ids=6 * A, w=7 * A, load=8 * A, ws=9 * A)
        a.update(kw)
        return L.moe_route_balanced(a["x"], B.MOE_BF16, 8, 256, a["wr"], a["lb"], a["sb"], ctypes.byref(p), a["lo"], a["ids"],
                                    a["w"], a["load"], a["ws"], need, None)

    outs, ins = ("ids", "w", "ws", "lo", "load"), ("x", "wr", "lb", "sb")
    for i, o in enumerate(outs):
        for other in outs[:i] + ins:
            assert balanced(**{o: 10 * A, other: 10 * A}) == bad, (o, other)

    def loss(l=A, load=2 * A, out=3 * A, d=4 * A, ws=5 * A):
        return L.moe_route_balance_loss(l, 100, load, ctypes.byref(p), 0.1, out, d, B.MOE_F32, 0, ws,
                                        B.moe_route_balance_loss_workspace_size(100, 64), None)

    for ws in (A, 2 * A, 3 * A, 4 * A):
        assert loss(ws=ws) == bad


def test_compilers_at_a_time(monkeypatch):
    from combine_dual_overlap_amd import build
    for value, want in (("3", 3), (" 2 ", 2), ("64", 8)):
        monkeypatch.setenv("MAX_JOBS", value)
        assert build.jobs() == want
    monkeypatch.delenv("MAX_JOBS")
    default = build.jobs()
    assert 1 <= default <= 8
    for value in ("", "0", "-2", "many", "1.5"):
        monkeypatch.setenv("MAX_JOBS", value)
        assert build.jobs() == default
