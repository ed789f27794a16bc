"""A role of the product kernels that gives up, as where a wait has run out: the others end too, the error is told, nothing is left behind.

Every kernel, by the sizes of test_project_plans_cpu.py.  No GPU fault is involved: the role stops by itself after its first chunk, and every
wait for it is bounded.
"""
import pytest
import torch

from tensor_train_compressed_mixed_b200 import TTEmbError, abi
from test_gpu_project import BF16, F16, F32, _randn, _table
from test_project_plans_cpu import CASES

pytestmark = pytest.mark.gpu
ROLES = {"copies": abi.TT_INJECT_COPIES, "products": abi.TT_INJECT_PRODUCTS, "sums": abi.TT_INJECT_SUMS}


@pytest.mark.parametrize("role", ROLES)
@pytest.mark.parametrize("product,kind,up,result,act,n,rows,dim,plan", CASES,
                         ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v).replace("torch.", ""))
def test_gives_up_and_recovers(role, product, kind, up, result, act, n, rows, dim, plan):
    g = torch.Generator(device="cuda").manual_seed(1)
    e, w = _table(rows, dim, kind, g, grad=torch.zeros(rows, dim, dtype=result, device="cuda"))
    x = _randn(g, n, dim, dtype=kind)
    dy = _randn(g, n, rows, dtype=up) if product else None
    pre = _randn(g, n, rows, dtype=kind) if product and act else None

    def call():
        if product == 0:
            return e.project(x, activation=act, out_dtype=result)
        out = torch.empty(n, dim, dtype=result, device="cuda") if product == 1 else False
        out = e.project_backward(x if product == 2 else None, dy, pre=pre, activation=act, grad_x=out, table_grad=product == 2)
        return e.grad.clone() if product == 2 else out
    want = call()
    e.sync()
    abi.tt_emb_dense_debug_inject(e.handle, ROLES[role])
    call()
    call()                                  # does nothing: the error waits
    with pytest.raises(TTEmbError) as err:
        e.sync()
    assert err.value.code == abi.TT_ERR_TIMEOUT
    got = call()                            # tensor memory is free, and the hook was consumed
    e.sync()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", [BF16, F32])
def test_the_calls_later_kernels_do_nothing(kind):
    n, rows, dim = 700, 2000, 520
    g = torch.Generator(device="cuda").manual_seed(2)
    e, w = _table(rows, dim, kind, g, grad=torch.full((rows, dim), 5.0, device="cuda"))
    x, dy, pre = _randn(g, n, dim, dtype=kind), _randn(g, n, rows, dtype=kind), _randn(g, n, rows, dtype=kind)
    gb = torch.full((rows,), 5.0, device="cuda")
    for role in ROLES.values():
        abi.tt_emb_dense_debug_inject(e.handle, role)
        e.project_backward(x, dy, pre=pre, activation="gelu", grad_bias=gb)         # x's gradient is the first product
        with pytest.raises(TTEmbError) as err:
            e.sync()
        assert err.value.code == abi.TT_ERR_TIMEOUT
        assert (e.grad == 5).all() and (gb == 5).all()
    abi.tt_emb_dense_debug_inject(e.handle, abi.TT_INJECT_COPIES)
    abi.tt_emb_dense_debug_inject(e.handle, abi.TT_INJECT_NONE)
    e.project_backward(x, dy, pre=pre, activation="gelu", grad_bias=gb)
    e.sync()
    assert not (e.grad == 5).any() and not (gb == 5).any()


@pytest.mark.parametrize("role", ROLES)
@pytest.mark.parametrize("kind,out,n,rows,dim", [(BF16, BF16, 4096, 8200, 4096), (BF16, F32, 2050, 8200, 1024), (F32, F32, 2050, 4100, 520), (F16, F16, 2050, 4200, 8200)])
def test_many_tiles(role, kind, out, n, rows, dim):
    """Blocks, and pairs of them, that have more tiles to come: the block whose partner has given up waits its own time."""
    g = torch.Generator(device="cuda").manual_seed(3)
    e, w = _table(rows, dim, kind, g)
    x = _randn(g, n, dim, dtype=kind)
    want = e.project(x, out_dtype=out)
    e.sync()
    abi.tt_emb_dense_debug_inject(e.handle, ROLES[role])
    e.project(x, out_dtype=out)
    with pytest.raises(TTEmbError) as err:
        e.sync()
    assert err.value.code == abi.TT_ERR_TIMEOUT
    assert torch.equal(e.project(x, out_dtype=out), want)
    e.sync()
