"""Few rows by tables that tensor maps cannot read as they lie: on either side of the rule that reads them by the FP32 pipes or lays them out.

Tolerances are those of test_gpu_project.py.
"""
import pytest
import torch

from test_gpu_project import BF16, F16, F32, STEP, _act64, _half_step, _inside, _least, _randn, _sum_tol, _table, _wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 3, 16, 17, 31, 32, 33])
@pytest.mark.parametrize("rows,dim", [(1, 4097), (130, 67), (1500, 130), (5844, 281), (12000, 1001), (20011, 515), (70001, 65)])
@pytest.mark.parametrize("kind,out,act", [(F32, F32, "silu"), (BF16, BF16, "gelu"), (F16, F32, None)])
def test_few_rows(n, rows, dim, kind, out, act):
    g = torch.Generator(device="cuda").manual_seed(n + rows)
    e, w = _table(rows, dim, kind, g)
    x, b, res = _randn(g, n, dim + 1, dtype=kind)[:, :dim], _randn(g, rows), _randn(g, n, rows, dtype=out)
    y, pre = _wide(n, rows, 3, out), _wide(n, rows, 1, F32)
    e.project(x, bias=b, activation=act, residual=res, out=y[:, :rows], pre=pre[:, :rows])
    e.sync()
    z = x.double() @ w.double().t() + b.double()
    tol = _sum_tol(x.double(), w.double().t(), dim) + 2 * STEP * z.abs()
    _inside(pre[:, :rows], z, tol + STEP * z.abs())
    want = _act64(act, z, None)
    tol = 1.13 * tol + (16 * STEP if out == F32 else 2.0 ** -15) * (want.abs() + 2.0 ** -100)
    want = want + res.double()
    tol = tol + STEP * want.abs()
    _inside(y[:, :rows], want, tol + _half_step(out) * (want.abs() + tol) + _least(out))
    assert (y[:, rows:] == 7).all() and (pre[:, rows:] == 7).all()
