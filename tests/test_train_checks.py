"""More checks of the training entry points, without a GPU: addresses are made up, nothing is enqueued."""
import ctypes

import pytest
import torch

A = 1 << 20       # aligned made-up address


def _B():
    from combine_dual_overlap_amd import binding
    binding.lib()
    return binding


def _tensor(B, i, **kw):
    """An entry with 8-bit states whose arrays lie apart from every other entry's: 4096 elements, 32 scales."""
    base = dict(param=(8 * i + 1) * A, grad=(8 * i + 2) * A, m=(8 * i + 3) * A, v=(8 * i + 4) * A,
                m_scale=(8 * i + 5) * A + 3, v_scale=(8 * i + 5) * A + 35, master=(8 * i + 6) * A, n=4096, param_dtype=1,
                grad_dtype=1, state_dtype=2)
    base.update(kw)
    return B.moe_adamw_tensor(*base.values())


def _status(B, *tensors):
    """The first refusal of the table's way to a step: building, checking, stepping."""
    t = (B.moe_adamw_tensor * len(tensors))(*tensors)
    host = torch.zeros(B.lib().moe_adamw_table_size(len(tensors)), dtype=torch.uint8)
    st = B.lib().moe_adamw_table_build(t, len(tensors), host.data_ptr(), host.numel())
    if st != B.MOE_OK:
        return st
    st = B.lib().moe_adamw_table_check(host.data_ptr())
    if st != B.MOE_OK:                                        # a step says the same, and enqueues nothing
        hp = B.adamw_params()
        assert B.lib().moe_adamw_step(host.data_ptr(), A, ctypes.byref(hp), A, None, None, None) == st
    return st


def test_adamw_table_refuses_overlapping_scales():
    """Scales shared by two moments or two tensors, or lying inside any other array, in any order of the tensors."""
    B = _B()
    bad = B.MOE_ERR_INVALID_ARG
    assert _status(B, *[_tensor(B, i) for i in range(50)]) == B.MOE_OK        # (m_scale and v_scale touch)
    assert _status(B, _tensor(B, 0, m_scale=5 * A, v_scale=5 * A)) == bad
    assert _status(B, _tensor(B, 0, m_scale=5 * A, v_scale=5 * A + 31)) == bad
    assert _status(B, _tensor(B, 0, m_scale=5 * A, v_scale=5 * A + 32)) == B.MOE_OK
    arrays = dict(param=(A, 8192), grad=(2 * A, 8192), m=(3 * A, 4096), v=(4 * A, 4096), m_scale=(5 * A + 3, 32),
                  v_scale=(5 * A + 35, 32), master=(6 * A, 16384))
    for name, (at, size) in arrays.items():
        for scale in ("m_scale", "v_scale"):
            for where, ok in ((at - 32, name != "v_scale"), (at - 31, False), (at + size // 2, False),
                              (at + size - 1, False), (at + size, name != "m_scale")):
                want = B.MOE_OK if ok else bad
                kw = {scale: where}
                assert _status(B, _tensor(B, 0), _tensor(B, 1, **kw)) == want, (name, kw)
                assert _status(B, _tensor(B, 1, **kw), _tensor(B, 2), _tensor(B, 0)) == want, (name, kw)
                if not name.endswith("scale"):                # its own tensor's arrays
                    assert _status(B, _tensor(B, 0, **kw)) == want, (name, kw)
                assert _status(B, _tensor(B, 0), _tensor(B, 1, n=0, **kw)) == B.MOE_OK
                fresh = dict(n=100, state_dtype=0, m_scale=None, v_scale=None)
                assert _status(B, _tensor(B, 0), _tensor(B, 1, **fresh)) == B.MOE_OK


def test_adamw_table_check_refuses_what_is_no_table():
    B = _B()
    check = B.lib().moe_adamw_table_check
    zeros = torch.zeros(512, dtype=torch.uint8)
    assert check(None) == check(zeros.data_ptr()) == B.MOE_ERR_INVALID_ARG
    assert check(zeros.data_ptr() + 8) == B.MOE_ERR_MISALIGNED


def _refused(match, device="cpu", **kw):
    """TrainLayer refuses the small fp32 (cid 1) or bf16 (cid 2) layer with these inputs changed, before it needs a GPU."""
    import workloads as W
    from combine_dual_overlap_amd import TrainLayer
    inp = W.make_inputs(W.get_config(kw.pop("cid", 2), small=True))
    inp.update({n: f(inp[n]) for n, f in kw.items()})
    with pytest.raises(ValueError, match=match):
        TrainLayer(inp, device=device)


def test_train_layer_refuses_weights_of_another_type_or_shape():
    """The kernels read every weight as the activations' type: a smaller one would be read behind its end."""
    half, full = (lambda t: t.to(torch.bfloat16)), (lambda t: t.float())
    for name in ("w_router", "w2"):
        _refused(name, cid=1, **{name: half})
        _refused(name, cid=2, **{name: full})
        _refused(name, **{name: lambda t: t.double()})
        for cut in (lambda t: t[:-1], lambda t: t[..., :-8], lambda t: t[None], lambda t: t.transpose(-1, -2)):
            _refused(name, **{name: cut})
    for cut in (lambda t: t[:-1], lambda t: t[..., :-8], lambda t: t[:, :-8]):
        _refused("w13", w13=cut)
    _refused("shared_w13", shared_w13=lambda ts: [t.float() for t in ts])
    _refused("shared_w2", shared_w2=lambda ts: [t.float() for t in ts])
    _refused("shared_w13", shared_w13=lambda ts: [t[..., :-8] for t in ts])
    _refused("shared_w2", shared_w2=lambda ts: [t[:-8] for t in ts])


def test_train_layer_refuses_tokens_on_another_device():
    """x and forced_ids are read by kernels of the layer's device (no GPU here: a layer without buffers, tensors
    without memory)."""
    from types import SimpleNamespace
    from combine_dual_overlap_amd import TrainLayer
    layer = object.__new__(TrainLayer)
    layer.cfg, layer.act, layer.T_max = SimpleNamespace(H=128, k=2), torch.bfloat16, 4
    layer.device, layer.forced_ids = torch.device("cuda", 0), None
    x = torch.empty(4, 128, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="x: .*cuda:0"):
        layer.forward(x)
    layer.device = torch.device("meta")
    with pytest.raises(ValueError, match="forced_ids: .*meta"):
        layer.forward(x, forced_ids=torch.zeros(4, 2, dtype=torch.int32))
    assert layer.T == 0


def test_workspace_query_of_sizes_without_a_product():
    """Sizes and types that moe_grouped_gemm refuses need no workspace, also where their tile counts leave 32 bits."""
    B = _B()
    top = (1 << 31) - 8
    ask = B.lib().moe_grouped_gemm_workspace_size
    assert ask(2, 1, 1, 1, 8192, 64, 64) > 0
    for kind in (0, 1, 2):
        for args in ((1, 1, 1, 64, top, 4096), (1, 1, 1, 64, 64, top), (1, 1, 1, 64, (1 << 22) + 8, 4096),
                     (1, 1, 1, 64, 64, (1 << 22) + 8), (1, 1, 1, (1 << 30) + 1, 64, 4096), (1, 1, 1, 1 << 62, 64, 64),
                     (0, 0, 256, 8192, top, top), (2, 1, 1, 8192, 64, 64), (-1, 1, 1, 8192, 64, 64),
                     (1, 1, 2, 8192, 64, 64), (1, 1, 1, 8192, 60, 64), (0, 1, 1, 8192, 64, 62)):
            assert ask(kind, *args) == 0, (kind, args)


def test_train_layer_refuses_gradient_types_that_backward_cannot_write():
    """fp32 activations have fp32 gradients; others were refused by the first backward() only, or by the optimizer."""
    import workloads as W
    from combine_dual_overlap_amd import TrainLayer
    for cid, dt in ((1, torch.bfloat16), (1, torch.float16), (2, torch.float16), (2, torch.float64)):
        with pytest.raises(ValueError, match="grad_dtype"):
            TrainLayer(W.make_inputs(W.get_config(cid, small=True)), device="cpu", grad_dtype=dt)
