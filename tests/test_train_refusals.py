"""Argument checks of the training entry points, without a GPU: each bad call
is refused before any device access (the addresses are made up), and the
binding refuses shapes and types that do not belong together."""
import ctypes

import pytest
import torch

A = 1 << 20       # aligned made-up address


def _B():
    from combine_dual_overlap_amd import binding
    binding.lib()
    return binding


def test_grouped_gemm_refusals():
    B = _B()
    f = B.lib().moe_grouped_gemm

    def call(kind=0, a=A, b=2 * A, ab=1, off=A, E=4, cap=100, N=64, K=64, c=3 * A, ct=1, acc=0, ws=None, n=0):
        return f(kind, a, b, ab, off, E, cap, N, K, c, ct, acc, ws, n, None)

    bad = B.MOE_ERR_INVALID_ARG
    for kw in (dict(kind=3), dict(kind=-1), dict(E=0), dict(E=257), dict(cap=-1), dict(N=0), dict(K=0), dict(K=-8),
               dict(off=None), dict(acc=2), dict(a=None), dict(b=None), dict(c=None), dict(c=A), dict(c=2 * A)):
        assert call(**kw) == bad, kw
    for kw in (dict(ab=2), dict(ct=2), dict(ab=0, ct=1), dict(cap=(1 << 30) + 1), dict(N=(1 << 22) + 8),
               dict(kind=0, cap=1 << 30, N=1 << 16)):
        assert call(**kw) == B.MOE_ERR_UNSUPPORTED, kw
    for kw in (dict(N=60), dict(K=12), dict(ab=0, ct=0, K=2), dict(a=A + 8), dict(b=2 * A + 2), dict(c=3 * A + 4),
               dict(off=A + 4)):
        assert call(**kw) == B.MOE_ERR_MISALIGNED, kw
    # no rows: nothing to do, for the row products
    assert call(cap=0) == B.MOE_OK and call(kind=1, cap=0) == B.MOE_OK
    # a product that is split needs its workspace
    need = B.lib().moe_grouped_gemm_workspace_size(2, 1, 1, 1, 8192, 64, 64)
    assert need > 0
    split = dict(kind=2, off=None, E=1, cap=8192)
    assert call(**split) == bad
    assert call(**split, ws=A, n=need - 1) == B.MOE_ERR_WORKSPACE
    assert call(**split, ws=A + 16, n=need) == B.MOE_ERR_MISALIGNED
    # sizes for which there is no product
    for args in ((3, 1, 1, 1, 8192, 64, 64), (2, 1, 0, 0, 8192, 64, 64), (2, 1, 1, 1, 0, 64, 64), (2, 1, 1, 1, 8192, 0, 64)):
        assert B.lib().moe_grouped_gemm_workspace_size(*args) == 0


def test_swiglu_refusals():
    B = _B()
    L = B.lib()

    def fwd(x=A, w=2 * A, act=1, off=A, E=4, cap=100, H=64, I=32, gu=3 * A, h=4 * A):
        return L.moe_grouped_swiglu(x, w, act, off, E, cap, H, I, gu, h, None)

    def bwd(dy=A, w=2 * A, gu=3 * A, act=1, off=A, E=4, cap=100, H=64, I=32, dgu=4 * A):
        return L.moe_grouped_swiglu_backward(dy, w, gu, act, off, E, cap, H, I, dgu, None)

    for f, outs in ((fwd, ("x", "w", "h")), (bwd, ("dy", "w", "gu", "dgu"))):
        for name in outs:
            assert f(**{name: None}) == B.MOE_ERR_INVALID_ARG, name
            assert f(**{name: 5 * A + 4}) == B.MOE_ERR_MISALIGNED, name
        assert f(off=None) == B.MOE_ERR_INVALID_ARG and f(E=300) == B.MOE_ERR_INVALID_ARG
        assert f(act=2) == B.MOE_ERR_UNSUPPORTED and f(I=36) == B.MOE_ERR_MISALIGNED and f(H=68) == B.MOE_ERR_MISALIGNED
        assert f(cap=0) == B.MOE_OK and f(cap=-1) == B.MOE_ERR_INVALID_ARG
    assert fwd(h=A) == fwd(gu=A) == fwd(gu=4 * A) == B.MOE_ERR_INVALID_ARG
    assert bwd(dgu=A) == bwd(dgu=2 * A) == B.MOE_ERR_INVALID_ARG


def test_combine_and_route_backward_refusals():
    B = _B()
    L = B.lib()

    def comb(d=A, y=2 * A, act=1, T=8, H=64, k=2, cap=16, inv=A, w=A, dy=3 * A, dw=4 * A):
        return L.moe_combine_backward(d, y, act, T, H, k, cap, inv, w, dy, dw, None)

    bad = B.MOE_ERR_INVALID_ARG
    for kw in (dict(T=-1), dict(H=0), dict(k=0), dict(k=17), dict(cap=-1), dict(d=None), dict(y=None), dict(inv=None),
               dict(w=None), dict(dy=None), dict(dw=None), dict(dy=A), dict(dy=2 * A), dict(dw=A)):
        assert comb(**kw) == bad, kw
    assert comb(act=2) == comb(T=1 << 26) == B.MOE_ERR_UNSUPPORTED
    assert comb(H=60) == comb(d=A + 8) == comb(dw=A + 4) == B.MOE_ERR_MISALIGNED
    assert comb(T=0) == B.MOE_OK

    p = B.route_params(64, 6)

    def route(l=A, T=8, ids=A, dw=A, params=p, dl=2 * A, dt=0):
        return L.moe_route_backward(l, T, ids, dw, ctypes.byref(params) if params else None, dl, dt, None)

    for kw in (dict(T=-1), dict(l=None), dict(ids=None), dict(dw=None), dict(params=None), dict(dl=None), dict(dl=A),
               dict(params=B.route_params(300, 6)), dict(params=B.route_params(4, 5))):
        assert route(**kw) == bad, kw
    assert route(dt=2) == route(T=1 << 26) == B.MOE_ERR_UNSUPPORTED
    assert route(l=A + 4) == route(dl=2 * A + 8) == B.MOE_ERR_MISALIGNED
    assert route(T=0) == B.MOE_OK


def _table(B, **kw):
    """(status, table bytes) of a table of one tensor."""
    t = (B.moe_adamw_tensor * 1)()
    base = dict(param=A, grad=2 * A, m=3 * A, v=4 * A, m_scale=None, v_scale=None, master=None, n=100,
                param_dtype=1, grad_dtype=1, state_dtype=0)
    base.update(kw)
    t[0] = B.moe_adamw_tensor(*base.values())
    host = torch.zeros(B.lib().moe_adamw_table_size(1), dtype=torch.uint8)
    return B.lib().moe_adamw_table_build(t, 1, host.data_ptr(), host.numel()), host


def test_adamw_table_refusals():
    B = _B()
    bad = B.MOE_ERR_INVALID_ARG
    for kw in (dict(n=-1), dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(m_scale=A),
               dict(state_dtype=2), dict(state_dtype=2, m_scale=A), dict(param_dtype=0, master=5 * A), dict(grad=A),
               dict(v=3 * A), dict(master=A)):
        assert _table(B, **kw)[0] == bad, kw
    for kw in (dict(param_dtype=2), dict(grad_dtype=2), dict(state_dtype=1), dict(n=(1 << 36) + 1)):
        assert _table(B, **kw)[0] == B.MOE_ERR_UNSUPPORTED, kw
    for kw in (dict(param=A + 8), dict(grad=2 * A + 2), dict(m=3 * A + 4), dict(v=4 * A + 4), dict(master=5 * A + 4)):
        assert _table(B, **kw)[0] == B.MOE_ERR_MISALIGNED, kw
    assert _table(B)[0] == _table(B, n=0)[0] == _table(B, state_dtype=2, m_scale=A + 1, v_scale=A + 3)[0] == B.MOE_OK
    t = (B.moe_adamw_tensor * 1)()
    build = B.lib().moe_adamw_table_build
    host = torch.zeros(4096, dtype=torch.uint8)
    assert B.lib().moe_adamw_table_size(0) == B.lib().moe_adamw_table_size(-3) == 0
    assert build(None, 1, host.data_ptr(), 4096) == build(t, 0, host.data_ptr(), 4096) == build(t, 1, None, 4096) == bad
    assert build(t, 1, host.data_ptr() + 8, 4000) == B.MOE_ERR_MISALIGNED
    assert build(t, 1, host.data_ptr(), B.lib().moe_adamw_table_size(1) - 1) == B.MOE_ERR_WORKSPACE


def test_adamw_table_refuses_overlapping_arrays():
    """An array that is updated twice, or read as a gradient while it is updated, in any order of the tensors."""
    B = _B()

    def tensor(i, **kw):
        base = dict(param=(8 * i + 1) * A, grad=(8 * i + 2) * A, m=(8 * i + 3) * A, v=(8 * i + 4) * A, m_scale=None,
                    v_scale=None, master=(8 * i + 5) * A, n=A // 4, param_dtype=1, grad_dtype=0, state_dtype=0)
        base.update(kw)
        return B.moe_adamw_tensor(*base.values())

    def build(*tensors):
        t = (B.moe_adamw_tensor * len(tensors))(*tensors)
        host = torch.zeros(B.lib().moe_adamw_table_size(len(tensors)), dtype=torch.uint8)
        return B.lib().moe_adamw_table_build(t, len(tensors), host.data_ptr(), host.numel())

    # A bytes hold n fp32 elements: m, v, grad and master touch, which is fine
    assert build(*[tensor(i) for i in range(60)]) == B.MOE_OK
    assert build(tensor(0), tensor(1, grad=2 * A)) == B.MOE_OK             # two tensors may read one gradient
    assert build(tensor(0), tensor(1, grad=6 * A)) == B.MOE_OK             # right behind the first one's master
    for kw in (dict(param=A), dict(param=A + 1024), dict(m=3 * A), dict(v=4 * A - 64), dict(master=5 * A), dict(m=A),
               dict(m=2 * A), dict(grad=3 * A), dict(grad=3 * A - 64), dict(grad=6 * A - 64), dict(grad=A + A // 2 - 64)):
        assert build(tensor(0), tensor(1, **kw)) == B.MOE_ERR_INVALID_ARG, kw
        assert build(tensor(1, **kw), tensor(2), tensor(0)) == B.MOE_ERR_INVALID_ARG, kw
        assert build(tensor(0), tensor(1, n=0, **kw)) == B.MOE_OK, kw      # nothing overlaps with nothing


def test_adamw_step_refusals():
    B = _B()
    status, host = _table(B)
    assert status == B.MOE_OK
    empty = _table(B, n=0)[1]

    def call(hp=None, table=host.data_ptr(), dev=A, step=A, lr=None, gs=None):
        hp = B.adamw_params(**(hp or {}))
        return B.lib().moe_adamw_step(table, dev, ctypes.byref(hp), step, lr, gs, None)

    bad = B.MOE_ERR_INVALID_ARG
    nan, inf = float("nan"), float("inf")
    for hp in (dict(lr=-1.0), dict(lr=nan), dict(lr=inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
               dict(beta2=nan), dict(eps=0.0), dict(eps=1e-40), dict(eps=inf), dict(weight_decay=-1.0),
               dict(weight_decay=inf)):
        assert call(hp=hp) == bad, hp
    zeros = torch.zeros(512, dtype=torch.uint8)
    for kw in (dict(table=None), dict(dev=None), dict(step=None), dict(table=zeros.data_ptr())):
        assert call(**kw) == bad, kw
    for kw in (dict(dev=A + 64), dict(step=A + 4), dict(lr=A + 4), dict(gs=A + 4), dict(table=host.data_ptr() + 8)):
        assert call(**kw) == B.MOE_ERR_MISALIGNED, kw
    assert call(table=empty.data_ptr()) == B.MOE_OK          # only an empty tensor: nothing is enqueued


def test_binding_refuses_shapes_and_types():
    B = _B()
    bf = torch.bfloat16
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt)
    off = z(4, dt=torch.int32)
    gemm = lambda *a, **k: B.moe_grouped_gemm(*a, **k)
    for args in (("tt", z(4, 8), z(3, 8, 8), off, z(4, 8)),             # no such kind
                 ("nt", z(4, 8), z(3, 8, 16), off, z(4, 8)),            # K differs
                 ("nt", z(4, 8), z(3, 8, 8), off, z(5, 8)),             # rows differ
                 ("nt", z(4, 8), z(3, 8, 8, dt=torch.float32), off, z(4, 8)),
                 ("nt", z(4, 8), z(3, 8, 8), None, z(4, 8)),            # one group, three experts
                 ("nt", z(4, 8), z(2, 8, 8), off, z(4, 8)),             # offsets of three experts
                 ("nt", z(4, 8), z(3, 8, 8), off.long(), z(4, 8)),
                 ("nn", z(4, 8), z(3, 16, 8), off, z(4, 16)),
                 ("tn", z(4, 8), z(5, 8), off, z(3, 8, 8)),
                 ("tn", z(4, 8), z(4, 16), off, z(3, 8, 8)),
                 ("nt", z(4, 8), z(3, 8, 8), off, z(4, 8))):            # on the CPU
        with pytest.raises(ValueError):
            gemm(*args)
    with pytest.raises(ValueError):
        B.moe_grouped_swiglu(z(4, 8), z(3, 32, 8), off, z(4, 8))
    with pytest.raises(ValueError):
        B.moe_grouped_swiglu(z(4, 8), z(3, 16, 8), off, z(4, 8), gu=z(4, 8))
    with pytest.raises(ValueError):
        B.moe_grouped_swiglu_backward(z(4, 8), z(3, 8, 8), z(4, 8), off, z(4, 16))
    with pytest.raises(ValueError):
        B.moe_combine_backward(z(4, 8), z(8, 16), z(8, dt=torch.int32), z(4, 2, dt=torch.float32), z(8, 16),
                               z(4, 2, dt=torch.float32))
    with pytest.raises(ValueError):
        B.moe_combine_backward(z(4, 8), z(8, 8), z(7, dt=torch.int32), z(4, 2, dt=torch.float32), z(8, 8),
                               z(4, 2, dt=torch.float32))
    with pytest.raises(ValueError):
        B.moe_route_backward(z(4, 64, dt=torch.float32), z(4, 5, dt=torch.int32), z(4, 5, dt=torch.float32),
                             B.route_params(64, 6), z(4, 64))
    f = torch.float32
    ok = dict(params=[z(8)], grads=[z(8)], m=[z(8, dt=f)], v=[z(8, dt=f)])
    for kw in (dict(grads=[z(9)]), dict(m=[z(8)]), dict(v=[z(9, dt=f)]), dict(params=[], grads=[], m=[], v=[]),
               dict(master=[z(8)]), dict(m_scale=[z(1, dt=torch.uint8)]), dict(grads=[z(8), z(8)]),
               dict(m=[z(8, dt=torch.uint8)], v=[z(8, dt=torch.uint8)]),
               dict(m=[z(8, dt=torch.uint8)], v=[z(8, dt=torch.uint8)], m_scale=[z(2, dt=torch.uint8)],
                    v_scale=[z(2, dt=torch.uint8)]), dict()):
        with pytest.raises(ValueError):
            B.moe_adamw_table(**{**ok, **kw})


def test_grouped_gemm_workspace_bound():
    """No call needs more than the bound that callers allocate once."""
    B = _B()
    import random
    r = random.Random(1)
    largest = 0
    for _ in range(20000):
        lg = lambda hi: int(2 ** r.uniform(0, hi))
        dense = r.random() < 0.4
        args = (r.randrange(3), r.choice([0, 1]), int(dense), 1 if dense else r.randint(1, 256), lg(20), 8 * lg(13), 8 * lg(13))
        largest = max(largest, B.lib().moe_grouped_gemm_workspace_size(*args))
    assert 8 << 20 < largest <= B.GEMM_MAX_WORKSPACE


def test_train_layer_refuses_what_it_cannot_train():
    import workloads as W
    from combine_dual_overlap_amd import TrainLayer
    inp = W.make_inputs(W.get_config(3, small=True))            # fp8 weights
    with pytest.raises(ValueError):
        TrainLayer(inp, device="cpu")
    inp = W.make_inputs(W.get_config(1))
    with pytest.raises(ValueError):
        TrainLayer(inp, device="cpu", states="int8")
