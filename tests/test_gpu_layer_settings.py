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
