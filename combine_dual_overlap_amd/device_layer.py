"""Device-side plumbing around dbo_moe_layer: uploads one layer's weights,
builds the moe_layer_desc, owns the workspace and output, and runs the layer
through the C ABI.  Memory and streams come from torch; every step of the
layer runs in libdbomoe.so.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as B


def _dev(t, device):
    return None if t is None else t.contiguous().to(device, non_blocking=False)


def concat_shared(shared_w13: list, shared_w2: list):
    """Several always-on SwiGLU experts as ONE expert: gate rows stacked, then
    up rows stacked ([sum I_i, H] each), down matrices side by side.  The sum
    of the experts' outputs equals this expert's output (a layout change of
    the weights, done once at load time)."""
    if not shared_w13:
        return None, None, 0
    gates, ups = [], []
    for w in shared_w13:
        I = w.shape[0] // 2
        gates.append(w[:I])
        ups.append(w[I:])
    w13 = torch.cat(gates + ups, dim=0).contiguous()
    w2 = torch.cat(list(shared_w2), dim=1).contiguous()
    return w13, w2, w2.shape[1]


def quantize_weights(w: torch.Tensor, device):
    """w [E, N, K] (bfloat16 or float32, CPU or device) as 8-bit integers with a scale per row: int8 [E, N, K] and
    float32 [E, N] on `device`, one expert's floats there at a time."""
    q = torch.empty(w.shape, dtype=torch.int8, device=device)
    s = torch.empty(w.shape[:-1], dtype=torch.float32, device=device)
    for e in range(w.shape[0]):
        B.moe_quant_int8_rows(_dev(w[e], device), q[e], s[e])
    return q, s


def block_of(inp: dict, act, H: int):
    """The entries of inp["block"], checked: pre_norm, post_norm, gate [H] (or None), scale, eps, residual."""
    block = inp.get("block")
    if block is None:
        return None
    b = dict(pre_norm=None, post_norm=None, gate=None, scale=1.0, eps=1e-6, residual=True)
    unknown = set(block) - set(b)
    if unknown:
        raise ValueError(f"block: unknown entries {sorted(unknown)}")
    b.update(block)
    for name in ("pre_norm", "post_norm", "gate"):
        if b[name] is not None and (b[name].dtype != act or b[name].shape != (H,)):
            raise ValueError(f"block {name}: {act} [{H}]")
    cfg = inp["cfg"]
    if cfg.expert_end - cfg.expert_begin != cfg.E and (b["post_norm"] is not None or b["residual"]):
        raise ValueError("block: a share of the experts gives a part of the layer's sum, which is normed and added to x "
                         "after the shares are summed (post_norm None, residual False)")
    return b


class DeviceLayer:
    """One MoE layer resident on the GPU.

    `inp` is a dict with x [T,H], w_router [E,H], logit_bias, forced_ids, w13,
    w2, w13_scale, w2_scale, shared_w13, shared_w2 (CPU or device tensors) and
    `cfg` with the routing fields (E, k, score, renormalize, n_groups,
    topk_groups, group_topn, routed_scale, expert_begin, expert_end, H, I).
    fp8_act: run the routed experts with fp8 activations (fp8 weights only).
    int8: run them in 8-bit integers; w13 and w2 are bfloat16 and are quantised
    here, with a scale per output channel.

    inp may also hold select_bias [E] float32, added to the scores when experts
    are chosen (not to their weights), and block, a dict that makes the layer a
    block of a model:  out = x + scale * gate * norm(layer(norm(x))).  Its entries:
    pre_norm and post_norm [H], weights of the norms before and after the layer
    (None: no norm); gate [H] (None: none); scale (1.0); eps (1e-6); residual (True).
    With a share of the experts: post_norm None and residual False.
    """

    def __init__(self, inp: dict, device: str = "cuda", T_max: int = None, fp8_act: bool = False, int8: bool = False):
        cfg = inp["cfg"]
        self.cfg = cfg
        d = torch.device(device)
        self.device = d
        self.x = _dev(inp["x"], d)
        self.w_router = _dev(inp["w_router"], d)
        self.logit_bias = _dev(inp.get("logit_bias"), d)
        self.forced_ids = _dev(inp.get("forced_ids"), d)
        if int8:
            if self.x.dtype != torch.bfloat16 or inp["w13"].dtype != torch.bfloat16 or inp["w2"].dtype != torch.bfloat16:
                raise ValueError("int8: bfloat16 activations and weights")
            self.w13, self.w13_scale = quantize_weights(inp["w13"], d)
            self.w2, self.w2_scale = quantize_weights(inp["w2"], d)
        else:
            self.w13 = _dev(inp["w13"], d)
            self.w2 = _dev(inp["w2"], d)
            self.w13_scale = _dev(inp.get("w13_scale"), d)
            self.w2_scale = _dev(inp.get("w2_scale"), d)
        if self.w13.dtype == torch.int8:
            E_loc = cfg.expert_end - cfg.expert_begin
            for name, w, s, shape in (("w13", self.w13, self.w13_scale, (E_loc, 2 * cfg.I, cfg.H)),
                                      ("w2", self.w2, self.w2_scale, (E_loc, cfg.H, cfg.I))):
                if (w.dtype != torch.int8 or w.dim() != 3 or w.shape[0] < E_loc or w.shape[1:] != shape[1:] or s is None or
                        s.dtype != torch.float32 or s.shape != w.shape[:2]):
                    raise ValueError(f"{name}: int8 {list(shape)}, {name}_scale: float32 {list(shape[:2])}")
        self.select_bias = _dev(inp.get("select_bias"), d)
        if self.select_bias is not None and (self.select_bias.dtype != torch.float32 or self.select_bias.shape != (cfg.E,)):
            raise ValueError(f"select_bias: float32 [{cfg.E}]")
        self.block = block_of(inp, self.x.dtype, cfg.H)
        sh13, sh2, shI = concat_shared(inp.get("shared_w13") or [], inp.get("shared_w2") or [])
        self.shared_w13, self.shared_w2 = _dev(sh13, d), _dev(sh2, d)
        self.route = B.route_params(cfg.E, cfg.k, cfg.score, cfg.renormalize, cfg.n_groups, cfg.topk_groups,
                                    cfg.group_topn, cfg.routed_scale)
        self.desc = B.moe_layer_desc(
            cfg.H, cfg.I, B.dtype_code(self.x), B.dtype_code(self.w13), self.route,
            cfg.expert_begin, cfg.expert_end, B.ptr(self.w_router), B.ptr(self.w13), B.ptr(self.w2),
            B.ptr(self.w13_scale), B.ptr(self.w2_scale), shI, B.ptr(self.shared_w13), B.ptr(self.shared_w2),
            int(bool(fp8_act)), B.ptr(self.select_bias), self._block_params())
        self.T = self.x.shape[0]
        self.T_max = T_max or self.T
        nbytes = B.moe_layer_workspace_size(self.desc, self.T_max)
        if nbytes == 0:
            raise B.MoEError(B.MOE_ERR_INVALID_ARG, "moe_layer_workspace_size")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=d)
        self.out = torch.empty_like(self.x)
        self.ctx = B.DboContext()
        self.comm = torch.cuda.Stream(device=d)

    def _block_params(self):
        """The block as the library takes it (kept: the description points at it)."""
        if self.block is None:
            return None
        b = self.block
        for name in ("pre_norm", "post_norm", "gate"):
            b[name] = _dev(b[name], self.device)
        post = B.moe_post_norm_params(B.ptr(b["post_norm"]), B.ptr(b["gate"]),
                                      B.MOE_GATE_NONE if b["gate"] is None else B.MOE_GATE_CHANNEL, b["scale"], b["eps"], None)
        self.block_params = B.moe_block_params(B.ptr(b["pre_norm"]), post, int(bool(b["residual"])))
        return ctypes.pointer(self.block_params)

    def run(self, schedule: str = "dbo", min_tokens_to_split: int = 2, split_at: int = -1,
            comm_cu_budget: int = 0, ffn_tile_m: int = 0, x=None, out=None, forced_ids=None):
        x = self.x if x is None else x
        out = self.out if out is None else out
        forced = self.forced_ids if forced_ids is None else forced_ids
        opts = B.dbo_opts(B.SCHEDULES[schedule], min_tokens_to_split, split_at, comm_cu_budget, ffn_tile_m)
        # the compute stream is the caller's current stream (also under graph
        # capture); the comm stream joins it through the layer's events
        compute = torch.cuda.current_stream(self.device)
        B.dbo_moe_layer(self.ctx, self.desc, x, out, opts, self.ws, compute, self.comm,
                        forced_ids=forced, logit_bias=self.logit_bias)
        return out

    def view(self, mb: int, name: str, dtype, shape, T: int = None):
        """A tensor view of microbatch mb's intermediate `name` inside the
        workspace (layout of a call with T tokens)."""
        off = B.moe_layer_workspace_layout(self.desc, self.T if T is None else T, mb)[name]
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty(0, dtype=dtype).element_size()
        return self.ws[off:off + nbytes].view(dtype).view(*shape)
