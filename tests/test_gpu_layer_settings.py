"""What the layers' own settings and timers say: expert times with shared experts beside integer ones, the optimizer's
hyperparameters, the balance of what was trained."""
import pytest
import torch

from test_gpu_block_layer import _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_ffn_times_hold_the_shared_experts_of_integer_layers():
    """The expert time of a layer with large shared experts beside small routed ones, eager and split."""
    import workloads as W
    from combine_dual_overlap_amd import DeviceLayer
    times = {}
    for n_shared in (0, 2):
        cfg = W.get_config(2, small=True).replace(T=4096, H=1024, I=64, k=2, n_shared=n_shared, shared_I=8192, wdt="bf16", act="bf16")
        layer = DeviceLayer(W.make_inputs(cfg, 5), int8=True)
        layer.run("unsplit")
        layer.ctx.set_timing(True)
        for schedule in ("unsplit", "serial"):
            whole, ffn = [], []
            for _ in range(7):
                a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
                a.record()
                layer.run(schedule)
                b.record()
                torch.cuda.synchronize()
                whole.append(a.elapsed_time(b))
                ffn.append(sum(layer.ctx.ffn_times(0)))
            times[n_shared, schedule] = sorted(whole)[3], sorted(ffn)[3]
    for schedule in ("unsplit", "serial"):
        (w0, f0), (w2, f2) = times[0, schedule], times[2, schedule]
        assert w2 > 1.5 * w0                       # they are most of this layer,
        assert f2 - f0 > 0.5 * (w2 - w0), (schedule, times)      # and the expert time grows by what the layer's does


def _train(**kw):
    from combine_dual_overlap_amd import TrainLayer
    cfg, inp = _inputs(1, "f32")
    layer = TrainLayer(inp, **kw)
    x = inp["x"].to(DEV)
    return layer, x, torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).to(DEV)


def test_the_norms_and_the_gate_follow_the_layers_hyperparameters():
    """layer.hyper changed between steps, as a schedule does: every weight takes it."""
    from combine_dual_overlap_amd import binding as B
    layer, x, dout = _train(lr=1e-2, weight_decay=0.0)

    def step():
        old = {n: w.clone() for n, w in layer.weights.items()}
        layer.forward(x)
        layer.backward(dout)
        layer.step()
        return {n: float((w - old[n]).abs().max()) for n, w in layer.weights.items()}

    layer.hyper.lr = 0.0
    assert set(step().values()) == {0.0}
    layer.hyper.lr = 1e-3
    # a step's m / sqrt(v) is at most (1 - beta1^2) / (1 - beta1) / ... = 1 where the gradients are alike; 2 leaves room
    assert all(0.0 < d < 2e-3 for d in step().values())
    layer.hyper = B.adamw_params(lr=0.0)
    assert set(step().values()) == {0.0}


def test_a_step_that_fails_half_way_keeps_the_count_of_what_was_done(monkeypatch):
    from combine_dual_overlap_amd import binding as B
    layer, x, dout = _train(lr=1e-2)
    real, calls = B.moe_adamw_step, []

    def fails(at):
        def call(*args, **kw):
            calls.append(1)
            if len(calls) == at:
                raise B.MoEError(B.MOE_ERR_HIP, "moe_adamw_step")
            return real(*args, **kw)
        return call

    for at, steps in ((1, 0), (2, 1)):
        calls.clear()
        layer.forward(x)
        layer.backward(dout)
        old = layer.weights["w2"].clone()
        monkeypatch.setattr(B, "moe_adamw_step", fails(at))
        with pytest.raises(B.MoEError):
            layer.step()
        monkeypatch.setattr(B, "moe_adamw_step", real)
        assert layer.steps.item() == steps and torch.equal(layer.weights["w2"], old) == (steps == 0)


def test_passes_that_are_not_trained_on_do_not_move_the_bias():
    """forward() for evaluation, then two that backward() follows: the bias goes by the tokens of these."""
    layer, x, dout = _train(lr=1e-3, bias_rate=0.125)
    bias, load = layer.select_bias.clone(), torch.zeros_like(layer.load)
    for i in range(6):
        layer.forward((x * (i + 1) - i).contiguous() if i not in (2, 4) else x)
        if i in (2, 4):
            load += layer.load
            with pytest.raises(ValueError):                # refused: not counted
                layer.backward(torch.stack([dout, dout], 2)[..., 0])
            layer.backward(dout)
    layer.step()
    want = bias + 0.125 * torch.sign(load.float().mean() - load.float())
    assert torch.equal(layer.select_bias, want)
    assert layer.load_sum.abs().sum() == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_balance_loss_does_not_change_the_choice_of_experts(score):
    """Softmax scores are not limited to groups without a selection bias, in training as in serving."""
    import workloads as W
    from combine_dual_overlap_amd import DeviceLayer, TrainLayer
    cfg = W.get_config(1, small=True).replace(k=3, n_groups=4, topk_groups=2, group_topn=1, score=score)
    inp = W.make_inputs(cfg, 5)
    inp["forced_ids"] = None
    x = inp["x"].to(DEV)
    plain, loss = TrainLayer(inp), TrainLayer(inp, balance_coef=0.1)
    want, got = plain.forward(x), loss.forward(x)
    ids = plain.buf["ids"][:cfg.T]
    assert torch.equal(loss.buf["ids"][:cfg.T], ids)
    # the weights are fp32's of one gate and 64 bits' of the other: a few half steps
    assert (got - want).abs().max() <= 2.0 ** -20 * want.abs().max()
    serve = DeviceLayer(inp)
    serve.run("unsplit")
    assert torch.equal(serve.view(0, "topk_ids", torch.int32, (cfg.T, cfg.k)), ids)
