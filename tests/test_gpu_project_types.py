"""Gradients of the table's projection where dz, the table and the results are of different types: over the whole range of dz's values,
and with no fewer bits of dz than the result has.

Tolerances are those of test_gpu_project.py: a sum of k products in fp32 is off by k + 2 steps of 2^-23 of the sum of magnitudes and
2^-22 for operands as terms, dz in fp32 by 32 steps, dz as two terms by 2^-17 of it, and a result is rounded once.  The two terms: a bf16
value of [2^e, 2^(e + 1)) has steps of 2^(e - 7), so the first leaves at most 2^(e - 8), and the second, whose steps are 2^(e - 16) for what is
below that, at most 2^(e - 17).
"""
import pytest
import torch

from test_gpu_project import BF16, F16, F32, STEP, _act64, _half_step, _inside, _least, _randn, _sum_tol, _table

pytestmark = pytest.mark.gpu


def _backward(n, rows, dim, kind, dy, gx, gw, act=None, extra=0, by=1.0, bias=False, seed=1):
    """One backward pass on a table of values about `by`, compared with 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    e, w = _table(rows, dim, kind, g, grad=torch.empty(rows, dim, dtype=gw, device="cuda"))
    w.copy_(_randn(g, rows, dim, dtype=kind, by=by))
    x = _randn(g, n, dim + extra, dtype=kind, by=by)[:, :dim]
    pre = _randn(g, n, rows, dtype=kind, by=3.0) if act else None
    cap = 2.5 if act == "softcap" else None
    gb = torch.empty(rows, device="cuda") if bias else None
    got = e.project_backward(x, dy, pre=pre, activation=act, cap=cap, grad_x=torch.empty(n, dim, dtype=gx, device="cuda"), grad_bias=gb)
    e.sync()
    d, off = dy.double(), torch.zeros(n, rows, dtype=torch.float64, device="cuda")
    if act:
        z = pre.double().requires_grad_()
        d, = torch.autograd.grad(_act64(act, z, cap), z, d)
        off = 32 * STEP * dy.double().abs()
    for got, a, o, b, k in ((got, d, off, w, rows), (e.grad, d.t(), off.t(), x, n)):
        want = a @ b.double()
        if kind != F32 and got.dtype != F32 and (act or dy.dtype == F32):       # dz as two terms
            o = o + 2.0 ** -17 * (a.abs() + o)
        if kind == got.dtype == BF16 and (act or dy.dtype != BF16):     # dz in as many bits as this result
            o = o + _half_step(BF16) * (a.abs() + o) + _least(BF16)
        tol = _sum_tol(a, b.double(), k) + o @ b.double().abs()
        _inside(got, want, tol + _half_step(got.dtype) * (want.abs() + tol) + _least(got.dtype))
    if bias:
        _inside(gb, d.sum(0), d.abs().sum(0) * (n + 4) * STEP + off.sum(0))


def _spread(n, rows, dtype, low, high, extra=0, seed=2):
    """Values of either sign, of magnitudes from 10^low to 10^high."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 10.0 ** (low + (high - low) * torch.rand(n, rows + extra, generator=g, device="cuda")) * torch.randn(n, rows + extra, generator=g, device="cuda").sign()
    return x.to(dtype)[:, :rows]


# by the tensor cores as they lie and copied, by few tiles and slices of k, and by the FP32 pipes
SIZES = [(200, 1000, 512, 0), (65, 129, 257, 3), (2050, 1030, 128, 8), (5, 30011, 64, 1), (7, 70, 40, 0), (1, 1, 1, 0), (4100, 3000, 1288, 0)]


@pytest.mark.parametrize("n,rows,dim,extra", SIZES)
@pytest.mark.parametrize("low,high,by", [(-9, 5, 1e-3), (-9, -7, 1.0), (4, 5, 1e-3), (-2, 2, 1.0)])
@pytest.mark.parametrize("result", [BF16, F16, F32])
def test_fp16_table_with_bf16_gradients(n, rows, dim, extra, low, high, by, result):
    """bf16 gradients go far beyond fp16's range on either side; the sums need not."""
    if result == F16:       # no fp16 result of a table this large leaves the type: sums of up to 4100 values
        by = min(by, 1.0 / 10.0 ** high)
    _backward(n, rows, dim, F16, _spread(n, rows, BF16, low, high, extra), result, result, extra=extra, by=by, bias=True)


@pytest.mark.parametrize("result", [BF16, F32])
@pytest.mark.parametrize("act", ["gelu", "softcap"])
def test_fp16_table_with_bf16_gradients_and_an_activation(act, result):
    for n, rows, dim, extra in ((200, 1000, 512, 0), (65, 129, 257, 3)):
        _backward(n, rows, dim, F16, _spread(n, rows, BF16, -9, 5, extra), result, result, act=act, extra=extra, by=1e-3, bias=True)


@pytest.mark.parametrize("up", [BF16, F16])
@pytest.mark.parametrize("kind,result", [(F32, F32), (F32, BF16), (BF16, F32), (F16, F32)])
def test_gradients_of_fewer_bits_than_the_table_or_the_result(kind, result, up):
    for n, rows, dim, extra in SIZES[:4]:
        _backward(n, rows, dim, kind, _spread(n, rows, up, -3, 1, extra), result, result, extra=extra, bias=True)


@pytest.mark.parametrize("act", ["gelu", "silu", "softcap", "relu"])
@pytest.mark.parametrize("low,high,by", [(-7, -5, 1.0), (4.6, 4.8, 1e-3)])
@pytest.mark.parametrize("result", [BF16, F16, F32])
def test_fp16_gradients_times_slopes_at_the_ends_of_the_range(act, low, high, by, result):
    """Small gradients times small slopes go below fp16's least value, and large ones times gelu's largest, 1.13, beyond its greatest."""
    if result == F16:
        by = min(by, 1e-4)
    for n, rows, dim, extra in SIZES:
        if (n, rows) != (1, 1):
            _backward(n, rows, dim, F16, _spread(n, rows, F16, low, high, extra), result, result, act=act, extra=extra, by=by, bias=True)


@pytest.mark.parametrize("act,up", [("gelu", BF16), ("silu", F16), ("softcap", F32), (None, F16), (None, F32)])
@pytest.mark.parametrize("gx,gw", [(F16, F16), (F16, BF16), (BF16, F16)])
def test_fp16_results_beside_a_bf16_table(act, up, gx, gw):
    """dz of eight bits would cost a result of eleven three of them."""
    for n, rows, dim, extra in SIZES:
        g = torch.Generator(device="cuda").manual_seed(3)
        dy = _randn(g, n, rows + extra, dtype=up)[:, :rows]
        _backward(n, rows, dim, BF16, dy, gx, gw, act=act, extra=extra, by=0.5, bias=True)
