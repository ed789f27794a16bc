"""Every kernel of the products against 64 bits, at the sizes for which test_project_plans_cpu.py shows that a whole B200 takes it.

Tolerances are those of test_gpu_project_types.py.
"""
import pytest
import torch

from test_gpu_project import BF16, F32, STEP, _act64, _half_step, _inside, _least, _randn, _sum_tol, _table
from test_project_plans_cpu import CASES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("product,kind,up,result,act,n,rows,dim,plan", CASES,
                         ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v).replace("torch.", ""))
def test_product(product, kind, up, result, act, n, rows, dim, plan):
    g = torch.Generator(device="cuda").manual_seed(n + rows + dim)
    e, w = _table(rows, dim, kind, g, grad=torch.full((rows, dim), 7.0, dtype=result, device="cuda") if product == 2 else None)
    x = _randn(g, n, dim, dtype=kind)
    off = 0.0
    if product == 0:
        got = e.project(x, activation=act, out_dtype=result)
        e.sync()
        a, b, k = x.double(), w.double().t(), dim
        want = _act64(act, a @ b, None)
    else:
        dy, pre = _randn(g, n, rows, dtype=up), _randn(g, n, rows, dtype=kind) if act else None
        buf = torch.full((n, dim), 7.0, dtype=result, device="cuda") if product == 1 else False
        got = e.project_backward(x if product == 2 else None, dy, pre=pre, activation=act, grad_x=buf, table_grad=product == 2)
        e.sync()
        d = dy.double()
        if act:
            d = torch.where(pre > 0, d, torch.zeros_like(d))          # relu
        if product == 2:
            got, a, b, k = e.grad, d.t(), x.double(), n
        else:
            a, b, k = d, w.double(), rows
        want = a @ b
        if kind != F32 and result != F32 and (act or up == F32):       # dz as two terms, or rounded to bf16
            off = 2.0 ** -17 if kind != BF16 or result != BF16 else _half_step(BF16)
    tol = _sum_tol(a, b, k) + off * (a.abs() @ b.abs()) + (2.0 ** -15 * want.abs() if product == 0 and act else 0.0)
    _inside(got, want, tol + _half_step(result) * (want.abs() + tol) + _least(result) + STEP * tol)
