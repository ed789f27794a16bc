"""Which buffers of one AdamW step may lie on one another: gradients among themselves, and nothing else."""
import ctypes

import pytest

from tensor_train_compressed_mixed_b200 import abi

MB = 1 << 20


def _create(tensors, bits=32, steps=900 * MB):
    recs = []
    for k, t in enumerate(tensors):
        kw = dict(param=(10 * k + 1) * MB, grad=(10 * k + 2) * MB, exp_avg=(10 * k + 3) * MB, exp_avg_sq=(10 * k + 4) * MB,
                  m_scale=(10 * k + 5) * MB, v_scale=(10 * k + 6) * MB, size=1000, param_type=abi.TT_F32, grad_type=abi.TT_F32)
        kw.update(t)
        recs.append(abi.AdamWTensor(**kw))
    h = ctypes.c_void_p(1)
    o = abi.AdamWOptions(beta1=0.9, beta2=0.999, eps=1e-8, state_bits=bits)
    rc = abi.lib().tt_emb_adamw_create(len(recs), (abi.AdamWTensor * len(recs))(*recs), ctypes.byref(o), steps, ctypes.byref(h))
    if h.value:
        abi.lib().tt_emb_adamw_destroy(h)
    return rc


@pytest.mark.parametrize("second", [
    dict(grad=1 * MB),                                                    # the first tensor's weights
    dict(grad=1 * MB + 3996), dict(grad=1 * MB - 3996), dict(grad=3 * MB), dict(grad=4 * MB + 4),
    dict(grad=11 * MB),                                                   # its own weights
    dict(grad=1 * MB + 3998, grad_type=abi.TT_BF16, size=1), dict(grad=1 * MB - 8, size=1 << 20),
    dict(grad=1 * MB - 1998, grad_type=abi.TT_F16),
])
def test_gradients_on_written_buffers_are_refused(second):
    assert _create([{}, second]) == abi.TT_ERR_ARG


@pytest.mark.parametrize("second", [dict(grad=5 * MB + 12), dict(grad=6 * MB), dict(grad=3 * MB + 996)])
def test_gradients_on_8_bit_state_are_refused(second):
    assert _create([{}, second], bits=8) == abi.TT_ERR_ARG


def test_the_step_count_on_another_buffer_is_refused():
    assert _create([{}], steps=3 * MB + 8) == abi.TT_ERR_ARG
    assert _create([{}], steps=2 * MB) == abi.TT_ERR_ARG


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("second", [
    {}, dict(grad=2 * MB), dict(grad=2 * MB + 100),                       # one gradient for both, or a part of it
    dict(grad=1 * MB + 4000), dict(grad=1 * MB - 4000), dict(grad=1 * MB, size=0), dict(grad=900 * MB + 8), dict(grad=900 * MB - 4000),
])
def test_other_buffers_side_by_side_are_not(second, bits):
    assert _create([{}, second], bits) in (abi.TT_OK, abi.TT_ERR_CUDA)    # the latter where there is no device
