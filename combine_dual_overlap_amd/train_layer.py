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
from .device_layer import block_of, concat_shared, _dev


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

    inp may hold "block", as for DeviceLayer: the layer is then x + scale * gate *
    norm(layer(norm(x))), and pre_norm, post_norm and gate [H] are weights like the
    others (names "pre_norm", "post_norm", "gate"; their gradients are float32 and
    they do not decay).

    Balance of the experts: inp["select_bias"] [E] float32 is added to the scores
    when experts are chosen; bias_rate > 0: step() moves it by bias_rate towards the
    experts that got fewer tokens than the mean in the passes since the last step that
    backward() followed (starting from zeros if it was not given); balance_coef > 0: backward() adds the gradient of the
    balance loss of its tokens, and balance_loss [1] holds that loss.  `load` [E]
    counts the tokens of the last forward() by expert.  Not with forced ids.

    With a share of the experts (cfg.expert_begin, expert_end) out, dx and the
    router's gradient are this share's part, to be summed over the shares (and those
    of the norm before the layer and of the gate); give the shared experts and the
    balance loss to one share only, or their part is counted more than once.
    """

    def __init__(self, inp: dict, device: str = "cuda", T_max: int = None, grad_dtype=torch.float32,
                 states: str = "f32", master: bool = True, balance_coef: float = 0.0, bias_rate: float = 0.0, **hyper):
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
        self.block = block_of(inp, act, H)
        self.n_decay = len(self.weights)      # what follows is not decayed
        if self.block is not None:
            for name in ("pre_norm", "post_norm", "gate"):
                if self.block[name] is not None:
                    self.weights[name] = own(name, self.block[name], H)
        if not (0.0 <= balance_coef < 3.4e38 and 0.0 <= bias_rate < 3.4e38):      # (fp32 numbers)
            raise ValueError("balance_coef and bias_rate: not negative, and finite")
        self.balance_coef, self.bias_rate = balance_coef, bias_rate
        self.select_bias = inp.get("select_bias")
        if self.select_bias is not None:
            if self.select_bias.dtype != torch.float32 or self.select_bias.shape != (cfg.E,):
                raise ValueError(f"select_bias: float32 [{cfg.E}]")
            self.select_bias = self.select_bias.contiguous().to(d, copy=True)
        elif bias_rate > 0:
            self.select_bias = torch.zeros(cfg.E, device=d)
        self.balanced = self.select_bias is not None or balance_coef > 0
        if self.balanced and self.forced_ids is not None:
            raise ValueError("forced_ids: not with a selection bias or a balance loss")
        # (without a selection bias a softmax gate has no groups; the balanced gate, which counts the load, has)
        groups = 1 if self.balanced and self.select_bias is None and cfg.score == "softmax" else cfg.n_groups
        self.route = B.route_params(cfg.E, cfg.k, cfg.score, cfg.renormalize, groups, cfg.topk_groups, cfg.group_topn,
                                    cfg.routed_scale)

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
        if self.balanced:
            self.load, self.load_sum = (torch.zeros(E, dtype=i32, device=d) for _ in range(2))
            self.balance_loss = torch.zeros(1, device=d)
            self.ws_balance = new(B.moe_route_balance_loss_workspace_size(T, E), dt=torch.uint8)
        if self.block is not None:
            self.buf.update(xn=new(T, H), y=new(T, H), dy_block=new(T, H), rstd_pre=new(T, dt=f32), rstd_post=new(T, dt=f32),
                            dx_block=new(T, H))
            self.ws_norm = new(B.moe_norm_backward_workspace_size(T, H), dt=torch.uint8)
        self.ws_route = new(max(B.moe_route_workspace_size(T, H, E), 256), dt=torch.uint8)
        self.ws_dispatch = new(max(B.moe_dispatch_workspace_size(T, k, E_loc), 256), dt=torch.uint8)
        self.ws_gemm = new(B.GEMM_MAX_WORKSPACE, dt=torch.uint8)      # whatever the number of tokens

        names = list(self.weights)
        self.grads = {name: torch.zeros(w.shape, dtype=grad_dtype if name in names[:self.n_decay] else f32, device=d)
                      for name, w in self.weights.items()}
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
        gs, n = list(self.grads.values()), self.n_decay

        def table(part):
            cols = (ws, gs, self.m, self.v, self.m_scale, self.v_scale, self.master)
            return B.moe_adamw_table(*(None if c is None else c[part] for c in cols))

        self.table = table(slice(0, n))
        self.hyper = B.adamw_params(**hyper)
        self.norm_table = table(slice(n, None)) if len(ws) > n else None
        self.steps = torch.zeros(1, dtype=i32, device=d)
        self.T = 0

    def _gemm(self, kind, a, b, offsets, c, accumulate=False):
        B.moe_grouped_gemm(kind, a, b, offsets, c, self.ws_gemm, accumulate=accumulate)
        return c

    def _rows(self, *names):
        """The parts of the buffers that a call of self.T tokens uses."""
        T, n = self.T, self.T * self.cfg.k
        per_token = {"logits", "ids", "w", "out", "dw", "dlogits", "dx_dense", "dx", "sh_gu", "sh_h", "sh_out", "sh_dgu",
                     "xn", "y", "dy_block", "rstd_pre", "rstd_post", "dx_block"}
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
        if forced is not None and self.balanced:
            raise ValueError("forced_ids: not with a selection bias or a balance loss")
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
        x = self._normed(x, True)
        if self.balanced:
            self.load.zero_()
            B.moe_route_balanced(x, W["w_router"], self.route, ids, w, self.ws_route, select_bias=self.select_bias,
                                 load=self.load, logits_out=logits, logit_bias=self.logit_bias)
        else:
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
        if self.block is None:
            B.moe_combine(y_perm, self.T, cfg.k, inv, w, out, shared_out=shared)
        else:
            b, (y, rstd) = self.block, self._rows("y", "rstd_post")
            B.moe_combine_post_norm(y_perm, inv, w, self.x if b["residual"] else None, out, b["eps"], W.get("post_norm"),
                                    W.get("gate"), b["scale"], shared_out=shared, y_out=y,
                                    rstd=rstd if "post_norm" in W else None)
        return out

    def _normed(self, x, compute=False):
        """What the layer computes from: x, or its norm."""
        if "pre_norm" not in self.weights:
            return x
        xn, rstd = self._rows("xn", "rstd_pre")
        if compute:
            B.moe_pre_norm(x, self.weights["pre_norm"], xn, self.block["eps"], rstd=rstd)
        return xn

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
        off, x, dblock = self.offsets, self._normed(self.x), dout
        if self.block is not None:
            y, dout, rstd = self._rows("y", "dy_block", "rstd_post")
            B.moe_post_norm_backward(dblock, y, dout, self.ws_norm, rstd if "post_norm" in W else None, W.get("post_norm"),
                                     G.get("post_norm"), W.get("gate"), G.get("gate"), self.block["scale"], more)
        B.moe_combine_backward(dout, y_perm, inv, w, dy, dw)
        self._gemm("tn", dy, h, off, G["w2"], more)
        B.moe_grouped_swiglu_backward(dy, W["w2"], gu, off, dgu)
        self._gemm("tn", dgu, x_perm, off, G["w13"], more)
        self._gemm("nn", dgu, W["w13"], off, dx_perm)
        B.moe_route_backward(logits, ids, dw, self.route, dlogits)
        if self.balance_coef > 0:
            B.moe_route_balance_loss(logits, self.load, self.route, self.balance_coef, self.balance_loss, dlogits,
                                     self.ws_balance, accumulate=True)
        self._gemm("tn", dlogits, x, None, G["w_router"], more)
        self._gemm("nn", dlogits, W["w_router"], None, dx_dense)
        if "shared_w13" in W:
            sh_gu, sh_h, sh_dgu = self._rows("sh_gu", "sh_h", "sh_dgu")
            self._gemm("tn", dout, sh_h, None, G["shared_w2"], more)
            B.moe_grouped_swiglu_backward(dout, W["shared_w2"], sh_gu, None, sh_dgu)
            self._gemm("tn", sh_dgu, x, None, G["shared_w13"], more)
            self._gemm("nn", sh_dgu, W["shared_w13"], None, dx_dense, True)
        B.moe_combine(dx_perm, self.T, self.cfg.k, inv, self.ones[:self.T], dx, shared_out=dx_dense)
        if self.block is not None:
            dx = self._block_dx(dx, dblock if self.block["residual"] else None, more)
        if self.bias_rate > 0:
            self.load_sum.add_(self.load)
        self.fresh = False
        return dx

    def _block_dx(self, dxn, dres, more):
        """The gradient of x from that of what the layer computed from, and the residual's."""
        W = self.weights
        out, rstd = self._rows("dx_block", "rstd_pre")
        if "pre_norm" in W:
            B.moe_pre_norm_backward(dxn, self.x, rstd, W["pre_norm"], out, self.grads["pre_norm"], self.ws_norm, dres=dres,
                                    accumulate=more)
        elif dres is not None:
            B.moe_post_norm(dxn, dres, out, self.block["eps"])       # their sum
        else:
            return dxn
        return out

    def _captured(self):
        self.captured = self.captured or torch.cuda.is_current_stream_capturing()
        return self.captured

    def zero_grad(self):
        with torch.cuda.device(self.device):
            self._captured()
            for g in self.grads.values():
                g.zero_()
        self.fresh = True

    def _norm_hyper(self):
        """Those of the norms and the gate: no decay, and another seed (the tables number their tensors from 0 each)."""
        h = self.hyper
        return B.adamw_params(h.lr, h.beta1, h.beta2, h.eps, 0.0, h.seed ^ 0x5bd1e995)

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
        if self.norm_table is not None:       # (what the first takes this takes too; after a failed launch the step counts)
            B.moe_adamw_step(self.norm_table, self._norm_hyper(), self.steps, lr_scale=lr_scale, grad_scale=grad_scale)
        if self.bias_rate > 0:
            B.moe_route_bias_update(self.select_bias, self.load_sum, self.bias_rate)
        self.zero_grad()
        self.T = 0                            # the weights are no longer those of the last forward pass
