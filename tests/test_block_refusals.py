"""Argument checks of the balanced gate, the 8-bit integer products and the norms, without a GPU: each bad call is
refused before any device access (the addresses are made up), and the binding refuses shapes and types that do not
belong together."""
import ctypes
import math

import pytest
import torch

A = 1 << 20       # aligned made-up address


def _B():
    from combine_dual_overlap_amd import binding
    binding.lib()
    return binding


def _expect(B, call, **by_status):
    for name, kws in by_status.items():
        want = {"bad": B.MOE_ERR_INVALID_ARG, "unsup": B.MOE_ERR_UNSUPPORTED, "mis": B.MOE_ERR_MISALIGNED,
                "ws": B.MOE_ERR_WORKSPACE, "ok": B.MOE_OK}[name]
        for kw in kws:
            assert call(**kw) == want, (name, kw)


def test_select_refusals():
    B = _B()
    p = B.route_params(64, 6)

    def call(l=A, T=8, b=2 * A, params=p, ids=3 * A, w=4 * A, load=5 * A):
        return B.lib().moe_route_select(l, T, b, ctypes.byref(params) if params else None, ids, w, load, None)

    _expect(B, call,
            bad=[dict(T=-1), dict(params=None), dict(l=None), dict(ids=None), dict(w=None), dict(w=A), dict(ids=A), dict(ids=4 * A),
                 dict(load=3 * A), dict(load=A), dict(params=B.route_params(300, 6)), dict(params=B.route_params(4, 5)),
                 dict(params=B.route_params(64, 17)), dict(params=B.route_params(64, 6, n_groups=7)),
                 dict(params=B.route_params(64, 20, n_groups=8, topk_groups=2)),
                 dict(params=B.route_params(64, 6, n_groups=8, topk_groups=9))],
            unsup=[dict(T=1 << 26)], mis=[dict(l=A + 4), dict(b=A + 8), dict(ids=A + 4), dict(w=A + 4), dict(load=A + 4)],
            ok=[dict(T=0), dict(T=0, l=None)])


def test_balanced_route_refusals():
    B = _B()
    p = B.route_params(64, 6)
    need = B.moe_route_workspace_size(8, 256, 64)

    def call(x=A, act=1, T=8, H=256, wr=2 * A, lb=None, sb=None, params=p, lo=None, ids=3 * A, w=4 * A, load=None, ws=5 * A, n=need):
        return B.lib().moe_route_balanced(x, act, T, H, wr, lb, sb, ctypes.byref(params) if params else None, lo, ids, w, load,
                                          ws, n, None)

    _expect(B, call, bad=[dict(T=-1), dict(H=0), dict(x=None), dict(wr=None), dict(ids=None), dict(w=None), dict(ws=None), dict(params=None)],
            unsup=[dict(act=2), dict(act=3), dict(H=192), dict(T=1 << 26)],
            mis=[dict(x=A + 2), dict(sb=A + 4), dict(lb=A + 4), dict(lo=A + 4), dict(load=A + 4), dict(ws=A + 16)],
            ws=[dict(n=need - 1)], ok=[dict(T=0)])


def test_bias_update_and_loss_refusals():
    B = _B()
    up = lambda b=A, l=2 * A, E=64, r=0.1: B.lib().moe_route_bias_update(b, l, E, r, None)
    _expect(B, up, bad=[dict(b=None), dict(l=None), dict(l=A), dict(E=0), dict(E=257), dict(r=-0.1), dict(r=math.nan), dict(r=math.inf)],
            mis=[dict(b=A + 4), dict(l=A + 4)])
    p = B.route_params(64, 6)
    need = B.moe_route_balance_loss_workspace_size(100, 64)

    def call(l=A, T=100, load=2 * A, params=p, coef=0.1, loss=3 * A, d=4 * A, dt=0, acc=0, ws=5 * A, n=need):
        return B.lib().moe_route_balance_loss(l, T, load, ctypes.byref(params) if params else None, coef, loss, d, dt, acc, ws, n, None)

    _expect(B, call, bad=[dict(T=-1), dict(acc=2), dict(coef=-1.0), dict(coef=math.nan), dict(loss=None), dict(l=None), dict(load=None),
                          dict(d=None), dict(ws=None), dict(d=A), dict(d=2 * A), dict(d=3 * A), dict(loss=A), dict(loss=2 * A), dict(ws=4 * A),
                          dict(params=None)],
            unsup=[dict(dt=2), dict(dt=3), dict(T=1 << 26)],
            mis=[dict(l=A + 4), dict(load=A + 4), dict(loss=A + 4), dict(d=A + 2), dict(ws=A + 16)], ws=[dict(n=need - 1)])
    for args in ((0, 64), (-1, 64), (5, 0), (5, 257)):
        assert B.moe_route_balance_loss_workspace_size(*args) == 0


def test_quant_and_dispatch_int8_refusals():
    B = _B()
    quant = lambda x=A, act=1, n=4, K=64, q=2 * A, s=3 * A: B.lib().moe_quant_int8_rows(x, act, n, K, q, s, None)
    _expect(B, quant, bad=[dict(n=-1), dict(K=0), dict(x=None), dict(q=None), dict(s=None), dict(q=A), dict(s=A), dict(s=2 * A)],
            unsup=[dict(act=2), dict(act=3)], mis=[dict(K=24), dict(x=A + 8), dict(q=A + 8), dict(s=A + 4)], ok=[dict(n=0)])
    need = B.moe_dispatch_workspace_size(10, 2, 8)

    def disp(x=A, act=1, T=10, H=128, ids=A, k=2, E=8, lo=0, hi=8, tm=0, cnt=A, off=A, to=None, perm=A, inv=A, q=2 * A, s=3 * A, ws=A,
             n=need):
        return B.lib().moe_dispatch_int8(x, act, T, H, ids, k, E, lo, hi, tm, cnt, off, to, perm, inv, q, s, ws, n, None)

    _expect(B, disp, bad=[dict(T=-1), dict(H=0), dict(k=0), dict(k=17), dict(E=0), dict(lo=-1), dict(hi=0), dict(hi=9), dict(to=A),
                          dict(x=None), dict(ids=None), dict(cnt=None), dict(off=None), dict(perm=None), dict(inv=None), dict(q=None),
                          dict(s=None), dict(ws=None)],
            unsup=[dict(act=2), dict(E=2000, hi=1500)],
            mis=[dict(H=24), dict(x=A + 4), dict(q=A + 8), dict(s=A + 4), dict(ws=A + 16)], ws=[dict(n=16)])


def test_int8_product_refusals():
    B = _B()
    L = B.lib()

    def gemm(a=A, asc=2 * A, b=3 * A, bsc=4 * A, off=A, E=4, cap=100, N=64, K=64, c=5 * A, ct=1):
        return L.moe_grouped_gemm_int8(a, asc, b, bsc, off, E, cap, N, K, c, ct, None)

    def swiglu(a=A, asc=2 * A, b=3 * A, bsc=4 * A, off=A, E=4, cap=100, N=64, K=64, c=5 * A, ct=1):
        return L.moe_grouped_swiglu_int8(a, asc, b, bsc, off, E, cap, K, N, c, ct, None)

    for f in (gemm, swiglu):
        _expect(B, f, bad=[dict(E=0), dict(E=257), dict(cap=-1), dict(N=0), dict(K=0), dict(off=None), dict(a=None), dict(asc=None),
                           dict(b=None), dict(bsc=None), dict(c=None), dict(c=A), dict(c=2 * A), dict(c=3 * A), dict(c=4 * A)],
                unsup=[dict(ct=2), dict(ct=3), dict(cap=(1 << 30) + 1), dict(N=(1 << 22) + 8), dict(K=(1 << 17) + 16),
                       dict(cap=1 << 30, N=1 << 16)],
                mis=[dict(N=60), dict(K=24), dict(a=A + 8), dict(asc=A + 4), dict(b=A + 8), dict(bsc=A + 4), dict(c=A + 4), dict(off=A + 4)],
                ok=[dict(cap=0)])
    assert swiglu(N=1 << 20, K=1 << 13) == B.MOE_ERR_UNSUPPORTED       # the up rows' offsets would pass 32 bits
    need = B.moe_ffn_int8_workspace_size(100, 64)
    assert need >= 100 * 64 * 5 + 400 and B.moe_ffn_int8_workspace_size(0, 64) == B.moe_ffn_int8_workspace_size(5, 0) == 0

    def ffn(x=A, xs=2 * A, H=128, I=64, off=A, E=4, cap=100, w13=3 * A, w2=4 * A, s13=5 * A, s2=6 * A, y=7 * A, ws=8 * A, n=need):
        return L.moe_grouped_ffn_int8(x, xs, H, I, off, E, cap, w13, w2, s13, s2, y, ws, n, None)

    _expect(B, ffn, bad=[dict(E=0), dict(off=None), dict(cap=-1), dict(H=0), dict(I=0)] + [{k: None} for k in
                        ("x", "xs", "w13", "w2", "s13", "s2", "y", "ws")] + [dict(y=v * A) for v in (1, 2, 3, 4, 5, 6, 8)],
            unsup=[dict(H=(1 << 17) + 16), dict(I=(1 << 17) + 16)],
            mis=[dict(H=136), dict(I=72), dict(x=A + 8), dict(y=A + 8), dict(ws=A + 16)], ws=[dict(n=need - 1)], ok=[dict(cap=0)])


def test_norm_refusals():
    B = _B()
    L = B.lib()
    pre = lambda x=A, act=1, T=8, H=64, w=2 * A, eps=1e-6, n=3 * A, r=None: L.moe_pre_norm(x, act, T, H, w, eps, n, r, None)
    sizes_bad = [dict(T=-1), dict(H=0)]
    sizes_unsup = [dict(act=2), dict(act=3), dict(H=32776), dict(act=0, H=16388), dict(T=1 << 22)]
    _expect(B, pre, bad=sizes_bad + [dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(x=None), dict(w=None), dict(n=None), dict(n=2 * A)],
            unsup=sizes_unsup, mis=[dict(H=60), dict(x=A + 8), dict(w=A + 8), dict(n=A + 8), dict(r=A + 4)], ok=[dict(T=0)])

    def params(post_w=2 * A, gate=None, gate_kind=0, scale=1.0, eps=1e-6, next_w=None):
        return B.moe_post_norm_params(post_w, gate, gate_kind, scale, eps, next_w)

    def post(y=A, act=1, T=8, H=64, res=4 * A, out=5 * A, r=None, nn=None, nr=None, q=True, **kw):
        return L.moe_post_norm(y, act, T, H, res, ctypes.byref(params(**kw)) if q else None, out, r, nn, nr, None)

    def comb(y=A, act=1, T=8, H=64, k=2, inv=A, w=A, sh=None, res=4 * A, out=5 * A, yo=None, r=None, nn=None, nr=None, q=True, **kw):
        return L.moe_combine_post_norm(y, act, T, H, k, inv, w, sh, res, ctypes.byref(params(**kw)) if q else None, out, yo, r, nn, nr, None)

    for f in (post, comb):
        _expect(B, f, bad=sizes_bad + [dict(q=None), dict(gate=A), dict(gate_kind=1), dict(gate=A, gate_kind=4), dict(eps=0.0), dict(scale=math.nan),
                                       dict(scale=math.inf), dict(next_w=A), dict(nn=A), dict(r=A, post_w=None), dict(nr=A), dict(y=None), dict(out=None),
                                       dict(out=A), dict(out=2 * A), dict(gate=5 * A, gate_kind=3), dict(next_w=6 * A, nn=A), dict(next_w=6 * A, nn=4 * A),
                                       dict(next_w=6 * A, nn=5 * A), dict(next_w=6 * A, nn=6 * A)],
                unsup=sizes_unsup, mis=[dict(H=60), dict(y=A + 8), dict(res=A + 8), dict(out=A + 8), dict(post_w=A + 8), dict(gate=A + 8, gate_kind=1),
                                        dict(next_w=A + 8, nn=7 * A), dict(next_w=6 * A, nn=7 * A + 8), dict(r=A + 4)], ok=[dict(T=0)])
    _expect(B, comb, bad=[dict(k=0), dict(k=17), dict(inv=None), dict(w=None), dict(sh=5 * A), dict(yo=A), dict(yo=4 * A), dict(yo=5 * A), dict(yo=2 * A)],
            mis=[dict(inv=A + 4), dict(w=A + 4), dict(sh=A + 8), dict(yo=6 * A + 8)])


def test_norm_backward_refusals():
    B = _B()
    L = B.lib()
    need = B.moe_norm_backward_workspace_size(8, 64)
    assert need > 0 and B.moe_norm_backward_workspace_size(0, 64) == B.moe_norm_backward_workspace_size(8, 0) == 0

    def pre(d=A, x=2 * A, act=1, T=8, H=64, r=3 * A, w=4 * A, dres=None, dx=5 * A, dw=6 * A, acc=0, ws=7 * A, n=need):
        return L.moe_pre_norm_backward(d, x, act, T, H, r, w, dres, dx, dw, acc, ws, n, None)

    def post(d=A, y=2 * A, act=1, T=8, H=64, r=3 * A, dy=5 * A, dw=6 * A, dg=None, acc=0, ws=7 * A, n=need, post_w=4 * A, gate=None,
             gate_kind=0, scale=1.0, eps=1e-6, next_w=None):
        q = B.moe_post_norm_params(post_w, gate, gate_kind, scale, eps, next_w)
        return L.moe_post_norm_backward(d, y, act, T, H, r, ctypes.byref(q), dy, dw, dg, acc, ws, n, None)

    _expect(B, pre, bad=[dict(T=-1), dict(H=0), dict(acc=2), dict(w=None), dict(d=None), dict(x=None), dict(r=None), dict(dx=None), dict(dx=2 * A),
                         dict(dx=4 * A), dict(dx=3 * A), dict(dw=5 * A), dict(dw=4 * A), dict(dw=3 * A), dict(dw=A), dict(dw=7 * A), dict(ws=None)],
            unsup=[dict(act=2), dict(H=32776), dict(T=1 << 22)],
            mis=[dict(H=60), dict(d=A + 8), dict(dres=A + 8), dict(dx=A + 8), dict(dw=A + 4), dict(ws=7 * A + 16)], ws=[dict(n=need - 1)])
    _expect(B, post, bad=[dict(T=-1), dict(acc=-1), dict(d=None), dict(y=None), dict(r=None), dict(dy=None), dict(dy=2 * A), dict(dw=5 * A),
                          dict(post_w=None), dict(post_w=None, dw=None), dict(dg=8 * A), dict(gate=8 * A, gate_kind=1, dg=8 * A),
                          dict(gate=8 * A, gate_kind=1, dg=6 * A), dict(gate=8 * A, gate_kind=0), dict(ws=None), dict(dw=4 * A)],
            unsup=[dict(act=3)], mis=[dict(gate=8 * A + 8, gate_kind=1), dict(gate=8 * A, gate_kind=1, dg=9 * A + 8)], ws=[dict(n=0)])


def test_binding_refuses_what_does_not_belong_together():
    B = _B()
    rp = B.route_params(8, 2)
    f = lambda *s: torch.zeros(*s)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    q = lambda *s: torch.zeros(*s, dtype=torch.int8)
    u = torch.zeros(1024, dtype=torch.uint8)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    calls = [
        lambda: B.moe_route_select(f(4, 9), rp, i(4, 2), f(4, 2)),
        lambda: B.moe_route_select(f(4, 8).double(), rp, i(4, 2), f(4, 2)),
        lambda: B.moe_route_select(f(4, 8), rp, f(4, 2), f(4, 2)),
        lambda: B.moe_route_select(f(4, 8), rp, i(4, 3), f(4, 2)),
        lambda: B.moe_route_select(f(4, 8), rp, i(4, 2), f(3, 2)),
        lambda: B.moe_route_select(f(4, 8), rp, i(4, 2), f(4, 2), select_bias=f(7)),
        lambda: B.moe_route_select(f(4, 8), rp, i(4, 2), f(4, 2), load=f(8)),
        lambda: B.moe_route_balanced(f(4, 128), bf(8, 128), rp, i(4, 2), f(4, 2), u),
        lambda: B.moe_route_balanced(f(4, 128), f(9, 128), rp, i(4, 2), f(4, 2), u),
        lambda: B.moe_route_balanced(f(4, 128), f(8, 128), rp, i(4, 2), f(4, 2), u, logits_out=f(4, 9)),
        lambda: B.moe_route_bias_update(f(8), i(7), 0.1),
        lambda: B.moe_route_bias_update(f(8), f(8), 0.1),
        lambda: B.moe_route_balance_loss(f(4, 8), i(7), rp, 0.1, f(1), f(4, 8), u),
        lambda: B.moe_route_balance_loss(f(4, 8), i(8), rp, 0.1, f(2), f(4, 8), u),
        lambda: B.moe_route_balance_loss(f(4, 8), i(8), rp, 0.1, f(1), f(4, 7), u),
        lambda: B.moe_quant_int8_rows(f(4, 16), q(4, 8), f(4)),
        lambda: B.moe_quant_int8_rows(f(4, 16), u[:64].view(4, 16), f(4)),
        lambda: B.moe_quant_int8_rows(f(4, 16), q(4, 16), f(5)),
        lambda: B.moe_dispatch_int8(f(4, 16), i(4, 2), 8, 0, 8, i(8), i(8), i(8), i(8), q(8, 16), f(8), u),
        lambda: B.moe_dispatch_int8(f(4, 16), i(4, 2), 8, 0, 8, i(8), i(9), i(8), i(8), q(7, 16), f(8), u),
        lambda: B.moe_dispatch_int8(f(4, 16), i(3, 2), 8, 0, 8, i(8), i(9), i(8), i(8), q(8, 16), f(8), u),
        lambda: B.moe_grouped_gemm_int8(q(4, 16), f(4), q(2, 8, 32), f(2, 8), i(3), f(4, 8)),
        lambda: B.moe_grouped_gemm_int8(q(4, 16), f(3), q(2, 8, 16), f(2, 8), i(3), f(4, 8)),
        lambda: B.moe_grouped_gemm_int8(q(4, 16), f(4), q(2, 8, 16), f(8), i(3), f(4, 8)),
        lambda: B.moe_grouped_gemm_int8(q(4, 16), f(4), q(2, 8, 16), f(2, 8), i(3), f(4, 16)),
        lambda: B.moe_grouped_gemm_int8(f(4, 16), f(4), q(2, 8, 16), f(2, 8), i(3), f(4, 8)),
        lambda: B.moe_grouped_swiglu_int8(q(4, 16), f(4), q(2, 8, 16), f(2, 8), i(3), f(4, 8)),
        lambda: B.moe_grouped_ffn_int8(q(4, 16), f(4), i(3), q(2, 32, 16), f(2, 32), q(2, 16, 16), f(2, 16), f(4, 16), u),
        lambda: B.moe_grouped_ffn_int8(q(4, 16), f(4), i(3), q(2, 16, 16), f(2, 16), q(2, 16, 16), f(2, 16), bf(4, 16), u),
        lambda: B.moe_pre_norm(f(4, 8), f(7), f(4, 8), 1e-6),
        lambda: B.moe_pre_norm(f(4, 8), bf(8), f(4, 8), 1e-6),
        lambda: B.moe_pre_norm(f(4, 8), f(8), bf(4, 8), 1e-6),
        lambda: B.moe_pre_norm(f(4, 8), f(8), f(4, 8), 1e-6, rstd=f(5)),
        lambda: B.moe_post_norm(f(4, 8), f(4, 7), f(4, 8), 1e-6),
        lambda: B.moe_post_norm(f(4, 8), f(4, 8), bf(4, 8), 1e-6),
        lambda: B.moe_combine_post_norm(f(8, 7), i(8), f(4, 2), None, f(4, 8), 1e-6),
        lambda: B.moe_combine_post_norm(f(8, 8), i(7), f(4, 2), None, f(4, 8), 1e-6),
        lambda: B.moe_combine_post_norm(f(8, 8), i(8), f(4, 2), None, f(4, 8), 1e-6, y_out=f(3, 8)),
        lambda: B.moe_pre_norm_backward(f(4, 8), f(4, 8), f(4), f(8), f(4, 8), f(7), u),
        lambda: B.moe_pre_norm_backward(f(4, 8), f(4, 8), f(4), f(8), f(4, 9), f(8), u),
        lambda: B.moe_post_norm_backward(f(4, 8), f(3, 8), f(4, 8), u),
        lambda: B.moe_post_norm_backward(f(4, 8), f(4, 8), f(4, 8), u, gate=f(7)),
        lambda: B.moe_post_norm_backward(f(4, 8), f(4, 8), f(4, 8), u, gate=f(8), dgate=f(4, 1)),
        lambda: B.moe_post_norm_backward(f(4, 8), f(4, 8), f(4, 8), u, dgate=f(8)),
        lambda: B.moe_post_norm_backward(bf(4, 8), bf(4, 8), bf(4, 8), u, gate=bf(4, 1)),
        # right shapes, but not on a device
        lambda: B.moe_pre_norm(f(4, 8), f(8), f(4, 8), 1e-6),
        lambda: B.moe_route_select(f(4, 8), rp, i(4, 2), f(4, 2)),
    ]
    for n, c in enumerate(calls):
        with pytest.raises(ValueError):
            c()
            print("accepted:", n)


def test_layer_description_refusals():
    """dbo_moe_layer's integer experts, selection bias and block."""
    B = _B()

    def size(block=None, post=None, **kw):
        d = B.moe_layer_desc(2048, 1408, B.MOE_BF16, B.MOE_INT8, B.route_params(64, 6), 0, 64, 256, 512, 768, 1024, 1280, 0, None, None)
        for k, v in kw.items():
            setattr(d, k, v)
        if block is not None or post is not None:
            q = B.moe_post_norm_params(256, 256, 1, 1.0, 1e-6, None)
            for k, v in (post or {}).items():
                setattr(q, k, v)
            b = B.moe_block_params(256, q, 1)
            for k, v in (block or {}).items():
                setattr(b, k, v)
            d.block = ctypes.pointer(b)
        return B.moe_layer_workspace_size(d, 64)

    n = size()
    assert n > 0 and size(select_bias=256) == n
    assert size(block={}) == n + 2 * 64 * 2048 * 2                     # the norm of each microbatch's tokens
    assert size(block=dict(pre_w=None)) == n
    for kw in (dict(act=B.MOE_F32), dict(H=2048 + 64), dict(I=1400), dict(w13_scale=None), dict(w2_scale=None), dict(fp8_act=1),
               dict(select_bias=260), dict(w13_scale=1028)):
        assert size(**kw) == 0, kw
    for kw in (dict(block=dict(pre_w=260)), dict(block=dict(residual=2)), dict(post=dict(eps=0.0)), dict(post=dict(next_w=256)),
               dict(post=dict(gate=None)), dict(post=dict(gate_kind=0)), dict(post=dict(gate_kind=4)), dict(post=dict(post_w=264))):
        assert size(**kw) == 0, kw


def test_block_entries_are_checked():
    from combine_dual_overlap_amd.device_layer import block_of
    from workloads import get_config
    cfg = get_config(2, small=True)
    w = torch.ones(cfg.H)
    ok = block_of(dict(cfg=cfg, block=dict(pre_norm=w)), torch.float32, cfg.H)
    assert ok["residual"] and ok["scale"] == 1.0 and ok["pre_norm"] is w and block_of(dict(cfg=cfg), torch.float32, cfg.H) is None
    share = cfg.replace(expert_end=8)
    for c, b in ((cfg, dict(norm=w)), (cfg, dict(pre_norm=w[:-1])), (cfg, dict(post_norm=w.bfloat16())), (cfg, dict(gate=w[None])),
                 (share, dict(pre_norm=w)), (share, dict(post_norm=w, residual=False))):
        with pytest.raises(ValueError):
            block_of(dict(cfg=c, block=b), torch.float32, cfg.H)
    assert block_of(dict(cfg=share, block=dict(pre_norm=w, residual=False)), torch.float32, cfg.H)
