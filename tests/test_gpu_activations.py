"""The activations and their slopes at every 16-bit value: far tails, clamps, zeros, infinities and NaN.

A table of one row with a single 1 gives z = x.  Results of 32 bits are within 16 steps of fp32 of the value, those of 16 bits within
2^-15 and their own rounding (test_gpu_project.py derives both), where the value is above 2^-100; smaller ones are off by 2^-100 at
most, as e^-w flushes to zero below 2^-126 and w is held at 100 (at 13 for gelu in 16 bits, where w Phi(-w) is below 2^-123).
Slopes are within 32 steps of fp32 of 1; those that are small are so relative to themselves, too: within 2^-15 beyond |z| = 4, where
they are products and quotients of exponentials, and differences only of terms of which one is at most 0.26 of the other.
"""
import math

import pytest
import torch

from tensor_train_compressed_mixed_b200 import DenseEmbedding
from test_gpu_project import BF16, F16, F32, STEP, _half_step, _least

pytestmark = pytest.mark.gpu
CAP = 2.5
FLOOR = 2.0 ** -100


def _every(kind):
    return torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(kind)


def _act(act, z):
    """In 64 bits; the normal distribution's tail by erfc, which keeps it."""
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return torch.where(z == -math.inf, 0.0, z * 0.5 * torch.special.erfc(-z / math.sqrt(2)))
    if act == "silu":
        return torch.where(z == -math.inf, 0.0, z / (1 + torch.exp(-z)))
    return CAP * torch.tanh(z / CAP)


def _slope(act, z):
    w = z.abs().clamp(max=1e4)
    if act == "relu":
        return torch.where(torch.isnan(z), z, (z > 0).double())
    if act == "gelu":
        tail = 0.5 * torch.special.erfc(w / math.sqrt(2)) - w * torch.exp(-w * w / 2) / math.sqrt(2 * math.pi)
    elif act == "silu":
        tail = torch.exp(-w) / (1 + torch.exp(-w)) * (1 - w / (1 + torch.exp(-w)))
    else:
        u = torch.exp(-2 * w / CAP)
        return torch.where(torch.isnan(z), z, 4 * u / (1 + u) ** 2)
    return torch.where(torch.isnan(z), z, torch.where(z > 0, 1 - tail, tail))


def _one(kind, dim):
    e = DenseEmbedding(1, dim, dtype=kind)
    w = torch.zeros(1, dim, dtype=kind, device="cuda")
    w[0, 0] = 1
    e.set_table(w, grad=torch.zeros(1, dim, device="cuda"))
    return e


# dim 1 runs on the FP32 pipes, dim 8 on the tensor cores
@pytest.mark.parametrize("dim", [1, 8])
@pytest.mark.parametrize("kind", [BF16, F16])
@pytest.mark.parametrize("act", ["relu", "gelu", "silu", "softcap"])
@pytest.mark.parametrize("out", [F32, BF16, F16])
def test_every_value(act, kind, dim, out):
    e = _one(kind, dim)
    x = torch.zeros(65536, dim, dtype=kind, device="cuda")
    x[:, 0] = _every(kind)
    y = e.project(x, activation=act, cap=CAP if act == "softcap" else None, out_dtype=out).view(-1)
    e.sync()
    want = _act(act, _every(kind).double())
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(y), nan)
    y, want = y[~nan].double(), want[~nan]
    near = want.to(out).double()
    far = torch.isinf(near)                                     # infinities, and values beyond the result's type
    assert torch.equal(y[far], near[far])
    y, want = y[~far], want[~far]
    tol = (16 * STEP if out == F32 else 2.0 ** -15) * want.abs() + FLOOR
    tol = tol + _half_step(out) * (want.abs() + tol) + _least(out)
    bad = (y - want).abs() > tol
    assert not bad.any(), (y[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dim", [1, 8])
@pytest.mark.parametrize("kind", [BF16, F16])
@pytest.mark.parametrize("act", ["relu", "gelu", "silu", "softcap"])
def test_every_slope(act, kind, dim):
    e = _one(kind, dim)
    z = _every(kind).view(-1, 1)
    dy = torch.ones(65536, 1, dtype=kind, device="cuda")
    gb = torch.zeros(1, device="cuda")
    gx = e.project_backward(None, dy, pre=z, activation=act, cap=CAP if act == "softcap" else None, table_grad=False,
                            grad_x=torch.full((65536, dim), 7.0, device="cuda"))
    e.sync()
    clean = ~torch.isnan(z.view(-1))
    assert not gx[clean][:, 1:].any()
    got, want = gx[:, 0].double(), _slope(act, z.view(-1).double())
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    got, want, at = got[clean], want[clean], z.view(-1).double()[clean]
    assert ((got - want).abs() <= 32 * STEP).all(), float((got - want).abs().max())
    small = (at.abs() > 4) & (want.abs() < 2.0 ** -3)
    off = (got - want).abs() - FLOOR
    assert (off[small] <= 2.0 ** -15 * want[small].abs()).all(), float((off[small] / want[small].abs().clamp(min=FLOOR)).max())
    ok = clean & torch.isfinite(z.view(-1))
    e.project_backward(None, dy[ok], pre=z[ok], activation=act, cap=CAP if act == "softcap" else None, table_grad=False, grad_x=False, grad_bias=gb)
    e.sync()
    total = _slope(act, z[ok].view(-1).double())
    assert abs(float(gb) - float(total.sum())) <= float((total.abs().sum() * 70000 * STEP) + 65536 * 32 * STEP)
