"""Host-side checks of the dense-table and AdamW entry points: what they refuse before any device work."""
import ctypes

import pytest
import torch

from tensor_train_compressed_mixed_b200 import AdamW, DenseEmbedding, abi

P = 4096          # an address that is only compared, never followed


@pytest.mark.parametrize("rows,dim,kind,pad,code", [
    (0, 4, abi.TT_F32, -1, abi.TT_ERR_SHAPE), (2 ** 31 - 1, 4, abi.TT_F32, -1, abi.TT_ERR_SHAPE),
    (4, 0, abi.TT_F32, -1, abi.TT_ERR_SHAPE), (4, 2 ** 20 + 1, abi.TT_F32, -1, abi.TT_ERR_SHAPE),
    (4, 4, 3, -1, abi.TT_ERR_ARG), (4, 4, -1, -1, abi.TT_ERR_ARG),
    (4, 4, abi.TT_F32, 4, abi.TT_ERR_SHAPE), (4, 4, abi.TT_F32, -2, abi.TT_ERR_SHAPE),
])
def test_dense_create_refuses_bad_tables(rows, dim, kind, pad, code):
    h = ctypes.c_void_p(1)
    assert abi.lib().tt_emb_dense_create(rows, dim, kind, 1.0, pad, ctypes.byref(h)) == code
    assert not h.value


def test_null_handles_are_refused():
    L = abi.lib()
    assert L.tt_emb_dense_create(4, 4, abi.TT_F32, 1.0, -1, None) == abi.TT_ERR_ARG
    assert L.tt_emb_dense_set_table(None, P, None, abi.TT_F32) == abi.TT_ERR_ARG
    assert L.tt_emb_dense_workspace_size(None, 4, ctypes.byref(ctypes.c_size_t())) == abi.TT_ERR_ARG
    assert L.tt_emb_dense_set_workspace(None, P, 4, 4) == abi.TT_ERR_ARG
    assert L.tt_emb_dense_forward(None, P, 8, 1, P, abi.TT_F32, 4, None) == abi.TT_ERR_ARG
    assert L.tt_emb_dense_backward(None, P, 8, 1, P, abi.TT_F32, 4, 0, None) == abi.TT_ERR_ARG
    assert L.tt_emb_dense_sync(None) == abi.TT_ERR_ARG
    assert L.tt_emb_dense_last_error(None) == abi.TT_ERR_ARG
    assert L.tt_emb_adamw_step(None, 0.1, None, None) == abi.TT_ERR_ARG
    assert abi.tt_emb_status_word(None) == 0 and abi.tt_emb_dense_status_word(None) == 0
    L.tt_emb_dense_destroy(None)
    L.tt_emb_adamw_destroy(None)


def _tensor(**kw):
    t = dict(param=P, grad=P, exp_avg=P, exp_avg_sq=P, m_scale=P, v_scale=P, size=10, param_type=abi.TT_F32,
             grad_type=abi.TT_F32, weight_decay=0.0)
    t.update(kw)
    return abi.AdamWTensor(**t)


def _create(tensor=None, count=1, steps=P, **kw):
    o = dict(beta1=0.9, beta2=0.999, eps=1e-8, state_bits=32)
    o.update(kw)
    h = ctypes.c_void_p(1)
    arr = (abi.AdamWTensor * 1)(tensor or _tensor())
    rc = abi.lib().tt_emb_adamw_create(count, arr, ctypes.byref(abi.AdamWOptions(**o)), steps, ctypes.byref(h))
    assert not h.value
    return rc


@pytest.mark.parametrize("kw", [
    dict(size=-1), dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None), dict(param=P + 2),
    dict(grad=P + 1, grad_type=abi.TT_BF16), dict(exp_avg=P + 2), dict(param_type=3), dict(grad_type=-1),
    dict(weight_decay=-0.1), dict(weight_decay=float("nan")), dict(weight_decay=1e300), dict(guard=P + 2),
])
def test_adamw_create_refuses_bad_tensors(kw):
    assert _create(_tensor(**kw)) == abi.TT_ERR_ARG


@pytest.mark.parametrize("kw", [
    dict(beta1=1.0), dict(beta2=-0.1), dict(beta1=float("nan")), dict(eps=0.0), dict(eps=1e-60), dict(eps=float("inf")),
    dict(state_bits=16), dict(reserved=1), dict(count=0), dict(steps=None), dict(steps=P + 4),
])
def test_adamw_create_refuses_bad_options(kw):
    assert _create(**kw) == abi.TT_ERR_ARG


def test_adamw_create_refuses_overlapping_buffers():
    h = ctypes.c_void_p(1)
    far = dict(exp_avg=2 * P, exp_avg_sq=3 * P, m_scale=4 * P, v_scale=5 * P)
    o = abi.AdamWOptions(beta1=0.9, beta2=0.999, eps=1e-8, state_bits=32)
    for a, b in ((_tensor(**far), _tensor(**{k: v * 64 for k, v in far.items()})),      # a parameter named twice
                 (_tensor(**far), _tensor(param=64 * P, exp_avg=2 * P + 36, exp_avg_sq=65 * P)),
                 (_tensor(exp_avg=2 * P, exp_avg_sq=2 * P), _tensor(size=0))):
        arr = (abi.AdamWTensor * 2)(a, b)
        assert abi.lib().tt_emb_adamw_create(2, arr, ctypes.byref(o), P, ctypes.byref(h)) == abi.TT_ERR_ARG


def test_adamw_8_bit_wants_scales():
    assert _create(_tensor(m_scale=None), state_bits=8) == abi.TT_ERR_ARG
    assert _create(_tensor(v_scale=P + 1), state_bits=8) == abi.TT_ERR_ARG


def test_python_classes_refuse_cpu_tensors_and_bad_lists():
    x = torch.zeros(4)
    with pytest.raises(TypeError):
        AdamW([x], [x])
    for bad in ([], [x]):
        with pytest.raises(ValueError):
            AdamW(bad, [])
    with pytest.raises(ValueError):
        AdamW([x], [x], weight_decay=[0.1, 0.2])
    with pytest.raises(ValueError):
        AdamW([x], [x], guards=[None, None])
    with pytest.raises(ValueError):
        AdamW([x], [x], state_bits=16)
    with pytest.raises(ValueError):
        DenseEmbedding(10, 4, padding_idx=10)
    with pytest.raises(TypeError):
        abi._tokens(torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        abi._rows(x, 1, 4, "out")
    with pytest.raises(TypeError):
        abi.dtype_code(torch.float64)
