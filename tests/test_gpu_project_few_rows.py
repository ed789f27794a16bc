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


# all three products of short sums, which the FP32 pipes take where operands would have to be laid out
@pytest.mark.parametrize("rows,cols,deep", [(33000, 4, 9), (4, 33000, 17), (520, 4100, 31), (4100, 520, 1), (33000, 4, 65), (9001, 70, 33), (70, 9001, 64),
                                            (100003, 3, 5), (1, 100003, 2)])
@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("act", [None, "silu"])
def test_short_sums(rows, cols, deep, kind, act):
    g = torch.Generator(device="cuda").manual_seed(rows + deep)
    e, w = _table(cols, deep, kind, g)
    x, res = _randn(g, rows, deep, dtype=kind), _randn(g, rows, cols)
    y = _wide(rows, cols, 3, F32)
    e.project(x, activation=act, residual=res, out=y[:, :cols])
    e.sync()
    want, tol = x.double() @ w.double().t(), _sum_tol(x.double(), w.double().t(), deep)
    want = _act64(act, want, None)
    tol = 1.13 * tol + 16 * STEP * (want.abs() + 2.0 ** -100) + STEP * (want + res.double()).abs()
    _inside(y[:, :cols], want + res.double(), tol + _least(F32))
    assert (y[:, cols:] == 7).all()
    # x's gradient: rows of dz of `deep` values by a table of that many rows; the table's: sums over `deep` rows of x
    for n, height, width in ((rows, deep, cols), (deep, rows, cols)):
        e, w = _table(height, width, kind, g, grad=torch.ones(height, width, device="cuda"))
        dy, x = _randn(g, n, height + 1, dtype=kind)[:, :height], _randn(g, n, width, dtype=kind)
        pre = _randn(g, n, height, dtype=kind) if act else None
        gx = e.project_backward(x, dy, pre=pre, activation=act, accumulate=True, grad_x=torch.empty(n, width, device="cuda"))
        e.sync()
        d, off = dy.double(), 0.0
        if act:
            z = pre.double().requires_grad_()
            d, = torch.autograd.grad(_act64(act, z, None), z, d)
            off = 32 * STEP
        _inside(gx, d @ w.double(), _sum_tol(d, w.double(), height) + off * (dy.double().abs() @ w.double().abs()) + _least(F32))
        want = d.t() @ x.double() + 1
        _inside(e.grad, want, _sum_tol(d.t(), x.double(), n) + off * (dy.double().abs().t() @ x.double().abs()) + STEP * want.abs())
