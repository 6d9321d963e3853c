"""MI355X-native Dual-Batch-Overlap expert-parallel MoE layer.

The compute path is libdbomoe.so (hand-written HIP kernels for gfx950 behind
the C ABI of include/dbomoe.h); `binding` exposes its entry points under the
same names, `device_layer` holds the device-side plumbing of one layer and
`train_layer` its training step.
"""
from . import binding
from .binding import (moe_route_topk, moe_dispatch, moe_grouped_ffn, moe_combine, dbo_moe_layer,
                      moe_grouped_gemm, moe_grouped_swiglu, moe_grouped_swiglu_backward, moe_combine_backward,
                      moe_route_backward, moe_adamw_table, moe_adamw_step, DboContext, MoEError)
from .device_layer import DeviceLayer
from .train_layer import TrainLayer

__all__ = ["binding", "moe_route_topk", "moe_dispatch", "moe_grouped_ffn", "moe_combine", "dbo_moe_layer",
           "moe_grouped_gemm", "moe_grouped_swiglu", "moe_grouped_swiglu_backward", "moe_combine_backward",
           "moe_route_backward", "moe_adamw_table", "moe_adamw_step", "DboContext", "MoEError", "DeviceLayer", "TrainLayer"]
