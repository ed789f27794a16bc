"""Long sums of terms of one sign, where what tensor cores cut off at each step adds up: results of 16 bits.

A sum is formed in tensor memory over 4096 k at most for fp16 results, 32768 for bf16: 256 or 2048 steps of 16, each of which cuts off at
most 2^-22 of it, 2^-14 or 2^-11 in all (the sums of those are added in fp32: below 2^-19).  A result is then rounded once, by half
the distance of its type's values there.
"""
import pytest
import torch

from tensor_train_compressed_mixed_b200 import DenseEmbedding
from test_gpu_project import BF16, F16

pytestmark = pytest.mark.gpu
CUT = {F16: 2.0 ** -14 + 2.0 ** -19, BF16: 2.0 ** -11 + 2.0 ** -19}
BITS = {F16: 11, BF16: 8}


def _check(got, want):
    """got near want, which is positive, by half a step and the cut."""
    kind = got.dtype
    want = want.double()
    half = torch.exp2(torch.floor(torch.log2(want)) - BITS[kind])
    off = ((got.double() - want).abs() - half) / want
    assert float(off.max()) <= CUT[kind], float(off.max())


def _terms(g, law, n, k, kind):
    """Rows of k positive values whose products with values about 1 have sums of about 16."""
    x = torch.rand(n, k, generator=g, device="cuda") + 0.5
    if law == "large first":        # the first 64 of k hold most of the sum
        x[:, 64:] *= 64 / k / 4
        x *= 0.2
    else:
        x *= 16 / k
    return x.to(kind)


def _near_one(g, n, k, kind):
    return (torch.rand(n, k, generator=g, device="cuda") + 0.5).to(kind)


@pytest.mark.parametrize("law", ["uniform", "large first"])
@pytest.mark.parametrize("kind,k", [(F16, 4096), (F16, 4160), (F16, 20011), (F16, 32768), (F16, 65536), (BF16, 32768), (BF16, 65536), (BF16, 70000)])
def test_projection(kind, k, law):
    n, rows = 2100, 4100            # so many tiles that none is shared, with ragged ends
    g = torch.Generator(device="cuda").manual_seed(k)
    w, x = _near_one(g, rows, k, kind), _terms(g, law, n, k, kind)
    e = DenseEmbedding(rows, k, dtype=kind)
    e.set_table(w, with_grad=False)
    y = e.project(x)
    e.sync()
    for r, c in ((slice(0, 40), slice(0, 300)), (slice(n - 40, n), slice(rows - 300, rows))):
        _check(y[r, c], x[r].double() @ w[c].double().t())


@pytest.mark.parametrize("kind,k", [(F16, 32000), (BF16, 65000)])
def test_gradients(kind, k):
    g = torch.Generator(device="cuda").manual_seed(5)
    n, dim = 2100, 2056             # x's gradient: a sum over the table's rows
    e = DenseEmbedding(k, dim, dtype=kind)
    w, dy = _near_one(g, k, dim, kind), _terms(g, "uniform", n, k, kind)
    e.set_table(w, with_grad=False)
    gx = e.project_backward(None, dy, table_grad=False)
    e.sync()
    _check(gx[-30:, -200:], dy[-30:].double() @ w[:, -200:].double())
    rows = 2050                     # the table's: a sum over rows of x
    e = DenseEmbedding(rows, dim, dtype=kind)
    e.set_table(w[:rows].contiguous(), grad=torch.empty(rows, dim, dtype=kind, device="cuda"))
    x, dy = _near_one(g, k, dim, kind), _terms(g, "uniform", rows, k, kind).t().contiguous()
    e.project_backward(x, dy, grad_x=False)
    e.sync()
    _check(e.grad[-30:, -200:], dy[:, -30:].double().t() @ x[:, -200:].double())
    # and added to what is there
    e.grad.fill_(16.0)
    e.project_backward(x, dy, grad_x=False, accumulate=True)
    e.sync()
    _check(e.grad[:30, :200], dy[:, :30].double().t() @ x[:, :200].double() + 16)


@pytest.mark.parametrize("kind", [F16, BF16])
def test_few_tiles(kind):
    """k shared by clusters of blocks and cut into slices: each adds a part of the same sums."""
    for n, rows, k in ((64, 256, 65536), (8, 32, 100000), (300, 700, 40000)):
        g = torch.Generator(device="cuda").manual_seed(n)
        w, x = _near_one(g, rows, k, kind), _terms(g, "large first", n, k, kind)
        e = DenseEmbedding(rows, k, dtype=kind)
        e.set_table(w, with_grad=False)
        y, pre = torch.empty(n, rows, dtype=kind, device="cuda"), torch.empty(n, rows, dtype=kind, device="cuda")
        e.project(x, out=y, pre=pre, activation="relu")
        e.sync()
        _check(y, x.double() @ w.double().t())
        assert torch.equal(y, pre)
