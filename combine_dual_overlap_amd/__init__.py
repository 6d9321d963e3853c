"""MI355X-native Dual-Batch-Overlap expert-parallel MoE layer.

The compute path is libdbomoe.so (hand-written HIP kernels for gfx950 behind
the C ABI of include/dbomoe.h); `binding` exposes its entry points under the
same names, `device_layer` holds the device-side plumbing of one layer and
`train_layer` its training step.
"""
from . import binding
from .binding import (moe_route_topk, moe_dispatch, moe_grouped_ffn, moe_combine, dbo_moe_layer,
                      moe_grouped_gemm, moe_grouped_swiglu, moe_grouped_swiglu_backward, moe_combine_backward,
                      moe_route_backward, moe_adamw_table, moe_adamw_step,
                      moe_route_select, moe_route_balanced, moe_route_bias_update, moe_route_balance_loss,
                      moe_quant_int8_rows, moe_dispatch_int8, moe_grouped_gemm_int8, moe_grouped_swiglu_int8,
                      moe_grouped_ffn_int8, moe_pre_norm, moe_post_norm, moe_combine_post_norm, moe_pre_norm_backward,
                      moe_post_norm_backward, DboContext, MoEError)
from .device_layer import DeviceLayer
from .train_layer import TrainLayer

__all__ = ["binding", "moe_route_topk", "moe_dispatch", "moe_grouped_ffn", "moe_combine", "dbo_moe_layer",
           "moe_grouped_gemm", "moe_grouped_swiglu", "moe_grouped_swiglu_backward", "moe_combine_backward",
           "moe_route_backward", "moe_adamw_table", "moe_adamw_step",
           "moe_route_select", "moe_route_balanced", "moe_route_bias_update", "moe_route_balance_loss",
           "moe_quant_int8_rows", "moe_dispatch_int8", "moe_grouped_gemm_int8", "moe_grouped_swiglu_int8",
           "moe_grouped_ffn_int8", "moe_pre_norm", "moe_post_norm", "moe_combine_post_norm", "moe_pre_norm_backward",
           "moe_post_norm_backward", "DboContext", "MoEError", "DeviceLayer", "TrainLayer"]
