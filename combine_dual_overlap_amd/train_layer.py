"""Training of one MoE layer on the GPU: forward pass that keeps what the
backward pass needs, backward pass, and the AdamW step, all through the C ABI.

Forward (the layer of dbo_moe_layer, unsplit): route, dispatch, gate/up with
SwiGLU, down projection, combine, and the always-on shared experts as one
dense group.  Backward runs the same steps in reverse; the dispatch's gradient
is a combine with unit weights.  The selection of experts has no gradient.
"""
from __future__ import annotations

import torch

from . import binding as B
from .device_layer import concat_shared, _dev


class TrainLayer:
    """One MoE layer with trainable weights (float32 or bfloat16, not fp8).

    `inp` is the dict DeviceLayer takes.  T_max: most tokens of a call.
    grad_dtype: type of the weights' gradients.  states: "f32", or "fp8" for
    8-bit optimizer states.  master: keep fp32 copies of bfloat16 weights (else
    they are rounded stochastically).  The remaining keywords are those of
    binding.adamw_params.

    forward(x) -> out [T, H]; backward(dout) -> dx [T, H], of the last forward(),
    adding to the gradients in `grads`; zero_grad() zeroes them; step() updates
    the weights and zeroes the gradients; the next backward() needs a new
    forward().  (The first backward() after either writes the gradients without
    reading them: what else was put there in between is replaced.)  Outputs live
    in the layer's buffers until the next call; x must stay as it is until
    backward().  Calls run on the current stream of the layer's device; calls of
    one layer on several streams need the caller's ordering.

    forward(), backward() and step() can be captured, each by itself or together;
    a replay is a call, in order with the others, on the same buffers and with the
    number of tokens and the x and dout it was captured with.  The host does not
    see replays: from the first capture on every backward() adds, step() no longer
    checks that a backward() came before it, and an eager backward() takes the
    tokens of the last forward() that was not a replay.

    With a share of the experts (cfg.expert_begin, expert_end) out, dx and the
    router's gradient are this share's part, to be summed over the shares; give the
    shared experts to one share only, or their part is counted more than once.
    """

    def __init__(self, inp: dict, device: str = "cuda", T_max: int = None, grad_dtype=torch.float32,
                 states: str = "f32", master: bool = True, **hyper):
        cfg = inp["cfg"]
        d = torch.device(device)
        if d.type == "cuda" and d.index is None:
            d = torch.device("cuda", torch.cuda.current_device())
        self.cfg, self.device = cfg, d
        act = inp["x"].dtype
        if act not in (torch.float32, torch.bfloat16) or inp["w13"].dtype != act:
            raise ValueError("trainable weights are float32 or bfloat16, in the activations' type")
        if grad_dtype not in (torch.float32, act):
            raise ValueError("grad_dtype: float32, or bfloat16 with bfloat16 weights")
        if states not in ("f32", "fp8"):
            raise ValueError("states: f32 or fp8")
        self.logit_bias, self.forced_ids = _dev(inp.get("logit_bias"), d), _dev(inp.get("forced_ids"), d)
        if self.logit_bias is not None and (self.logit_bias.dtype != torch.float32 or self.logit_bias.numel() != cfg.E):
            raise ValueError(f"logit_bias: float32 [{cfg.E}]")
        if cfg.E % (8 if act == torch.bfloat16 else 4):
            raise ValueError("the number of experts must be a multiple of 8 (float32: 4)")
        self.act, self.T_max = act, T_max or inp["x"].shape[0]
        sh13, sh2, shI = concat_shared(inp.get("shared_w13") or [], inp.get("shared_w2") or [])
        H, I, E_loc = cfg.H, cfg.I, cfg.expert_end - cfg.expert_begin

        def own(name, t, *shape):             # trained in place
            if t.dtype != act or t.shape != shape:
                raise ValueError(f"{name}: {act} {list(shape)}")
            return t.contiguous().to(d, copy=True)

        self.weights = {"w_router": own("w_router", inp["w_router"], cfg.E, H)[None],
                        "w13": own("w13", inp["w13"], E_loc, 2 * I, H), "w2": own("w2", inp["w2"], E_loc, H, I)}
        if shI:
            self.weights["shared_w13"] = own("shared_w13", sh13, 2 * shI, H)[None]
            self.weights["shared_w2"] = own("shared_w2", sh2, H, shI)[None]
        self.route = B.route_params(cfg.E, cfg.k, cfg.score, cfg.renormalize, cfg.n_groups, cfg.topk_groups,
                                    cfg.group_topn, cfg.routed_scale)

        k, E, T = cfg.k, cfg.E, self.T_max
        n = T * k
        new = lambda *shape, dt=act: torch.empty(shape, dtype=dt, device=d)
        i32, f32 = torch.int32, torch.float32
        self.buf = dict(logits=new(T, E, dt=f32), ids=new(T, k, dt=i32), w=new(T, k, dt=f32), counts=new(E_loc, dt=i32),
                        perm=new(n, dt=i32), inv=new(n, dt=i32), x_perm=new(n, H), gu=new(n, 2 * I), h=new(n, I),
                        y_perm=new(n, H), out=new(T, H), dy_perm=new(n, H), dw=new(T, k, dt=f32), dgu=new(n, 2 * I),
                        dx_perm=new(n, H), dlogits=new(T, E), dx_dense=new(T, H), dx=new(T, H))
        self.offsets = new(E_loc + 1, dt=i32)
        self.ones = torch.ones(T, k, device=d)
        if shI:
            self.buf.update(sh_gu=new(T, 2 * shI), sh_h=new(T, shI), sh_out=new(T, H), sh_dgu=new(T, 2 * shI))
        self.ws_route = new(max(B.moe_route_workspace_size(T, H, E), 256), dt=torch.uint8)
        self.ws_dispatch = new(max(B.moe_dispatch_workspace_size(T, k, E_loc), 256), dt=torch.uint8)
        self.ws_gemm = new(B.GEMM_MAX_WORKSPACE, dt=torch.uint8)      # whatever the number of tokens

        self.grads = {name: torch.zeros(w.shape, dtype=grad_dtype, device=d) for name, w in self.weights.items()}
        self.fresh = True                     # the gradients are zero
        self.captured = False                 # calls were captured: `fresh` says nothing any more
        ws = list(self.weights.values())
        self.master = [w.float() for w in ws] if act == torch.bfloat16 and master else None
        if states == "fp8":
            codes = lambda: [torch.zeros(w.numel(), dtype=torch.float8_e4m3fn, device=d) for w in ws]
            scales = lambda: [torch.zeros((w.numel() + 127) // 128, dtype=torch.uint8, device=d) for w in ws]
            self.m, self.v, self.m_scale, self.v_scale = codes(), codes(), scales(), scales()
        else:
            self.m, self.v = ([torch.zeros(w.numel(), device=d) for w in ws] for _ in range(2))
            self.m_scale = self.v_scale = None
        self.table = B.moe_adamw_table(ws, list(self.grads.values()), self.m, self.v, self.m_scale, self.v_scale,
                                       self.master)
        self.hyper = B.adamw_params(**hyper)
        self.steps = torch.zeros(1, dtype=i32, device=d)
        self.T = 0

    def _gemm(self, kind, a, b, offsets, c, accumulate=False):
        B.moe_grouped_gemm(kind, a, b, offsets, c, self.ws_gemm, accumulate=accumulate)
        return c

    def _rows(self, *names):
        """The parts of the buffers that a call of self.T tokens uses."""
        T, n = self.T, self.T * self.cfg.k
        per_token = {"logits", "ids", "w", "out", "dw", "dlogits", "dx_dense", "dx", "sh_gu", "sh_h", "sh_out", "sh_dgu"}
        return [self.buf[s][:T if s in per_token else n] for s in names]

    def forward(self, x, forced_ids=None):
        cfg = self.cfg
        self.T = 0                            # backward() refuses after a forward pass that failed
        if (x.dtype != self.act or x.dim() != 2 or x.shape[1] != cfg.H or not 0 < x.shape[0] <= self.T_max or
                x.device != self.device):
            raise ValueError(f"x: [T, {cfg.H}] of {self.act} on {self.device}, 1 <= T <= {self.T_max}")
        forced = self.forced_ids if forced_ids is None else forced_ids
        if forced is not None and (forced.dtype != torch.int32 or forced.dim() != 2 or forced.shape[0] < x.shape[0] or
                                   forced.shape[1] != cfg.k or forced.device != self.device):
            raise ValueError(f"forced_ids: int32 [{x.shape[0]}, {cfg.k}] on {self.device}")
        self.T, self.x = x.shape[0], x
        try:
            with torch.cuda.device(self.device):
                return self._forward(x, forced)
        except Exception:
            self.T = 0
            raise

    def _forward(self, x, forced):
        cfg, W = self.cfg, self.weights
        logits, ids, w, perm, inv, x_perm, gu, h, y_perm, out = self._rows(
            "logits", "ids", "w", "perm", "inv", "x_perm", "gu", "h", "y_perm", "out")
        B.moe_route_topk(x, W["w_router"], self.route, ids, w, self.ws_route, logits_out=logits,
                         logit_bias=self.logit_bias, forced_ids=forced)
        B.moe_dispatch(x, ids, cfg.E, cfg.expert_begin, cfg.expert_end, self.buf["counts"], self.offsets, perm, inv,
                       x_perm, self.ws_dispatch)
        B.moe_grouped_swiglu(x_perm, W["w13"], self.offsets, h, gu=gu)
        self._gemm("nt", h, W["w2"], self.offsets, y_perm)
        shared = None
        if "shared_w13" in W:
            sh_gu, sh_h, shared = self._rows("sh_gu", "sh_h", "sh_out")
            B.moe_grouped_swiglu(x, W["shared_w13"], None, sh_h, gu=sh_gu)
            self._gemm("nt", sh_h, W["shared_w2"], None, shared)
        B.moe_combine(y_perm, self.T, cfg.k, inv, w, out, shared_out=shared)
        return out

    def backward(self, dout):
        if self.T == 0:
            raise RuntimeError("backward() follows forward(), with the weights it used")
        if dout.shape != (self.T, self.cfg.H) or dout.dtype != self.act:
            raise ValueError(f"dout: [{self.T}, {self.cfg.H}] of {self.act}")
        with torch.cuda.device(self.device):
            return self._backward(dout)

    def _backward(self, dout):
        W, G, more = self.weights, self.grads, self._captured() or not self.fresh
        logits, ids, w, inv, x_perm, gu, h, y_perm, dy, dw, dgu, dx_perm, dlogits, dx_dense, dx = self._rows(
            "logits", "ids", "w", "inv", "x_perm", "gu", "h", "y_perm", "dy_perm", "dw", "dgu", "dx_perm", "dlogits",
            "dx_dense", "dx")
        off = self.offsets
        B.moe_combine_backward(dout, y_perm, inv, w, dy, dw)
        self._gemm("tn", dy, h, off, G["w2"], more)
        B.moe_grouped_swiglu_backward(dy, W["w2"], gu, off, dgu)
        self._gemm("tn", dgu, x_perm, off, G["w13"], more)
        self._gemm("nn", dgu, W["w13"], off, dx_perm)
        B.moe_route_backward(logits, ids, dw, self.route, dlogits)
        self._gemm("tn", dlogits, self.x, None, G["w_router"], more)
        self._gemm("nn", dlogits, W["w_router"], None, dx_dense)
        if "shared_w13" in W:
            sh_gu, sh_h, sh_dgu = self._rows("sh_gu", "sh_h", "sh_dgu")
            self._gemm("tn", dout, sh_h, None, G["shared_w2"], more)
            B.moe_grouped_swiglu_backward(dout, W["shared_w2"], sh_gu, None, sh_dgu)
            self._gemm("tn", sh_dgu, self.x, None, G["shared_w13"], more)
            self._gemm("nn", sh_dgu, W["shared_w13"], None, dx_dense, True)
        B.moe_combine(dx_perm, self.T, self.cfg.k, inv, self.ones[:self.T], dx, shared_out=dx_dense)
        self.fresh = False
        return dx

    def _captured(self):
        self.captured = self.captured or torch.cuda.is_current_stream_capturing()
        return self.captured

    def zero_grad(self):
        with torch.cuda.device(self.device):
            self._captured()
            for g in self.grads.values():
                g.zero_()
        self.fresh = True

    def step(self, lr_scale=None, grad_scale=None):
        """One AdamW update from the gradients added since zero_grad(); lr_scale, grad_scale: device scalars."""
        if self.fresh and not self.captured:
            raise RuntimeError("step() follows backward()")
        self.steps.add_(1)
        try:
            B.moe_adamw_step(self.table, self.hyper, self.steps, lr_scale=lr_scale, grad_scale=grad_scale)
        except Exception:
            self.steps.sub_(1)                # refused: no update has been made
            raise
        self.zero_grad()
        self.T = 0                            # the weights are no longer those of the last forward pass
