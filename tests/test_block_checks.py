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
