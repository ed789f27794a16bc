"""fp32 operands as bf16 terms: sums of one product each, which show every term and pair of terms that a result is made of.

A 24-bit value is t0 + t1 + t2 with t1 at most 2^-8 and t2 at most 2^-17 of it.  By a power of two every product of terms is exact, and so are their
sums: the result has all 24 bits.  By another 24-bit value the pairs that are left out, t1 u2, t2 u1 and t2 u2, are 2^-24 of the product,
the sums of the small pairs are cut by 5 steps of 2^-22 of 2^-7 of it, and the last sum is rounded by 2^-24: 2^-22 in all.  A
lost third term would be off by up to 2^-17, a lost t1 u1 by up to 2^-16.
"""
import pytest
import torch

from tensor_train_compressed_mixed_b200 import DenseEmbedding
from test_gpu_project import F32, STEP

pytestmark = pytest.mark.gpu


def _values(g, *shape):
    """Values of 24 random bits and some exponents."""
    x = 1 + torch.rand(*shape, generator=g, device="cuda", dtype=torch.float64)
    x = x * torch.exp2(torch.randint(-3, 4, shape, generator=g, device="cuda").double())
    return (x * (torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1)).float()


def _scale(g, n, powers):
    if not powers:
        return _values(g, n)
    return torch.exp2(torch.randint(-5, 6, (n,), generator=g, device="cuda").float())


def _same(got, want, powers):
    want = want.double()
    if powers:
        assert torch.equal(got.double(), want)
    else:
        assert ((got.double() - want).abs() <= 2.0 ** -22 * want.abs()).all(), float(((got.double() - want).abs() / want.abs().clamp(min=1e-30)).max())


# heights of 16 to 128 rows, single blocks and pairs, shared and sliced k, rows that tensor maps can take and others
@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("n,size", [(7, 1032), (33, 515), (100, 800), (300, 520), (1000, 1999), (4100, 264), (5000, 2100), (40, 6000)])
def test_every_term_of_fp32_operands(n, size, powers):
    g = torch.Generator(device="cuda").manual_seed(n)
    place = torch.randperm(size, generator=g, device="cuda")              # row c of the table holds one value, in column place[c]
    s = _scale(g, size, powers)
    w = torch.zeros(size, size, device="cuda")
    w[torch.arange(size, device="cuda"), place] = s
    e = DenseEmbedding(size, size)
    e.set_table(w, grad=torch.empty(size, size, device="cuda"))
    x, dy = _values(g, n, size), _values(g, n, size)
    y = e.project(x)
    gx = e.project_backward(None, dy, table_grad=False)
    e.sync()
    _same(y, x.double()[:, place] * s.double(), powers)
    _same(gx[:, place], dy.double() * s.double(), powers)
    # the table's gradient: each column of dy holds one value, in row at[c]
    at = torch.randint(n, (size,), generator=g, device="cuda")
    one = torch.zeros(n, size, device="cuda")
    one[at, torch.arange(size, device="cuda")] = s
    e.project_backward(x, one, grad_x=False)
    e.sync()
    _same(e.grad, x.double()[at] * s.double()[:, None], powers)


@pytest.mark.parametrize("k", [8192, 65536])
def test_long_sums_of_one_sign_in_fp32(k):
    """Chunks of 256 k: 16 steps, each of which cuts off up to 2^-22 of the chunk's sum, and their sums added in fp32, by half a step each.  Whole
    sums of 8192 k would be off by 4.8e-5."""
    from test_gpu_project import BF16, F16
    n, rows = 2100, 2100
    g = torch.Generator(device="cuda").manual_seed(k)
    for kind in (F16, BF16, F32):
        if kind == F32 and k > 8192:
            continue
        w = (torch.rand(rows, k, generator=g, device="cuda") + 0.5).to(kind)
        x = ((torch.rand(n, k, generator=g, device="cuda") + 0.5) * (16 / k)).to(kind)
        e = DenseEmbedding(rows, k, dtype=kind)
        e.set_table(w, with_grad=False)
        y = e.project(x, out_dtype=F32)
        e.sync()
        want = x[-50:].double() @ w[-300:].double().t()
        tol = 16 * 2.0 ** -22 + k / 256 * STEP / 2 + (2.0 ** -22 if kind == F32 else 0.0)
        assert ((y[-50:, -300:].double() - want).abs() <= tol * want).all(), float(((y[-50:, -300:].double() - want).abs() / want).max())
