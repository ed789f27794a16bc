"""Clipping of short lists, which sums and scales the gradients in one launch: again and again on what the call before wrote.

A clipped gradient is off by the norm's 18 half steps of fp32, the factor's, the product's and its type's half step (test_gpu_norm.py);
each further call adds as much, and its bound is chosen from the norm that the one before left in 64 bits.
"""
import pytest
import torch

from tensor_train_compressed_mixed_b200 import GradNorm
from test_gpu_norm import BF16, F16, F32, NORM_TOL, U, _half_step, _least, _lists, _norm64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [F32, BF16, F16])
@pytest.mark.parametrize("sizes", [[5], [1, 1000, 33], [16384] * 3, [70001]], ids=str)
@pytest.mark.parametrize("shift", [0, 3])
def test_clipped_again_without_a_pause(kind, sizes, shift):
    _, grads = _lists([kind], sizes, shift, by=0.5)
    o = GradNorm(grads)
    norm, was = _norm64(grads), [x.double() for x in grads]
    bounds = [norm * 0.8 ** (i + 1) for i in range(6)]
    seen = [o.clip(b).clone() for b in bounds]
    for i, got in enumerate(seen):
        want = norm if i == 0 else bounds[i - 1]
        # the rounding of 16-bit values to their type moves each by half a step at most, and so their norm
        assert abs(float(got) - want) <= ((i + 1) * (NORM_TOL + 4 * U) + i * _half_step(kind)) * want, (i, float(got), want)
    for x, a in zip(grads, was):
        want = a * 0.8 ** 6
        off = 6 * (NORM_TOL + 4 * U) + 15 * _half_step(kind)       # each call's rounding, and those that its norm saw
        assert ((x.double() - want).abs() <= off * want.abs() + 6 * _least(kind)).all()
