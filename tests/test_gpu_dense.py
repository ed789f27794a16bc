"""DenseEmbedding against the definition in 64 bits: sizes, types, strides, runs of equal tokens, refusals.

Tolerances count roundings: a lookup is one product in fp32 and one rounding to the output's
type; a gradient of k terms is at most k + 2 roundings in fp32 of the sum of magnitudes (k - 1
additions, the scale, the accumulation) and one to the gradient's type.  A rounding is off by
eps / 2 of the value, or by half the least subnormal.
"""
import numpy as np
import pytest
import torch

from tensor_train_compressed_mixed_b200 import DenseEmbedding, abi

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _least(dtype):
    return torch.finfo(dtype).smallest_normal * _half_step(dtype)


def _make(rows, dim, table, scale=1.0, pad=None, grad=None, seed=1):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(rows, dim, generator=g).to(table)
    e = DenseEmbedding(rows, dim, dtype=table, scale=scale, padding_idx=pad)
    buf = None if grad is None else torch.randn(rows, dim, generator=g).to(grad).cuda()
    e.set_table(w.cuda(), grad=buf, with_grad=grad is not None)
    return e, w


def _wide(rows, dim, extra, dtype, fill=7.0):
    return torch.full((rows, dim + extra), fill, dtype=dtype, device="cuda")


@pytest.mark.parametrize("n,rows,dim,table,out,ids,extra", [
    (1, 1, 1, F32, F32, torch.int64, 0), (3, 5, 8, BF16, BF16, torch.int32, 0), (33, 100, 64, F32, BF16, torch.int64, 8),
    (257, 300, 129, F32, F32, torch.int32, 0), (1000, 77, 1000, F16, F32, torch.int64, 3), (64, 50, 4096, BF16, BF16, torch.int64, 0),
    (4099, 200, 24, BF16, F16, torch.int32, 5), (5, 9, 8200, F32, F16, torch.int64, 8), (20000, 1000, 7, F16, F16, torch.int64, 1),
    (3000, 400, 2056, BF16, F32, torch.int64, 0),
])
def test_lookup(n, rows, dim, table, out, ids, extra):
    e, w = _make(rows, dim, table, scale=3.7)
    tok = torch.randint(rows, (n,), generator=torch.Generator().manual_seed(n)).to(ids)
    buf = _wide(n, dim, extra, out)
    got = e.forward(tok.cuda(), out=buf[:, :dim])
    e.sync()
    want = w[tok.long()].double() * float(np.float32(3.7))
    tol = (_half_step(out) + U) * (1 + U) * want.abs() + _least(out)
    assert (got.double().cpu() - want).abs().sub(tol).max() <= 0
    assert (buf[:, dim:] == 7.0).all()


def test_lookup_shapes_and_empty_calls():
    e, w = _make(10, 4, F32, grad=F32)
    tok = torch.tensor([[1, 9, 0], [3, 3, 3]], device="cuda")
    assert torch.equal(e.forward(tok).cpu(), w[tok.cpu()])
    assert e.forward(tok, out_dtype=BF16).dtype == BF16
    assert e.forward(torch.tensor(7, device="cuda")).shape == (4,)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert e.forward(none).shape == (0, 4)
    before = e.grad.clone()
    e.backward(none, torch.empty(0, 4, device="cuda"), accumulate=True)
    assert torch.equal(e.grad, before)
    e.backward(none, torch.empty(0, 4, device="cuda"))
    e.sync()
    assert not e.grad.any()


def _check_grad(e, tok, up, before, scale, pad, out, stride0=False):
    """e.grad against sums in 64 bits, within the counted roundings."""
    rows, dim = e.num_rows, e.dim
    t = tok.cpu().long().reshape(-1)
    u = up.double().cpu().reshape(-1, dim)
    keep = torch.ones_like(t, dtype=torch.bool) if pad is None else t != pad
    s = float(np.float32(scale))
    want = torch.zeros(rows, dim, dtype=torch.float64).index_add_(0, t[keep], u[keep]) * s
    size = torch.zeros(rows, dim, dtype=torch.float64).index_add_(0, t[keep], u[keep].abs()) * abs(s)
    if before is not None:
        want, size = want + before, size + before.abs()
    k = torch.bincount(t[keep], minlength=rows).double()[:, None]
    tol = (k + 2) * U * 1.01 * size + _half_step(out) * (1 + 1e-3) * want.abs() + _least(out)
    err = (e.grad.double().cpu() - want).abs()
    assert err.sub(tol).max() <= 0, float((err - tol).max())
    if before is None:
        assert not e.grad[k.cuda()[:, 0] == 0].any()      # rows no token names


LAWS = {
    "uniform": lambda n, r, g: torch.randint(r, (n,), generator=g),
    "same": lambda n, r, g: torch.full((n,), r // 2),
    "sorted": lambda n, r, g: torch.arange(n) % r,
    "runs": lambda n, r, g: (torch.arange(n) // 32) % r,          # runs that end where tiles do
    "few": lambda n, r, g: torch.randint(min(r, 3), (n,), generator=g),
}


@pytest.mark.parametrize("law", sorted(LAWS))
@pytest.mark.parametrize("n,rows,dim,up,out,extra,accumulate", [
    (1, 1, 1, F32, F32, 0, False), (32, 7, 8, BF16, BF16, 0, False), (33, 100, 17, F32, F32, 3, True),
    (64, 3, 520, F16, F32, 8, False), (1000, 501, 129, F32, BF16, 0, False), (5000, 300, 64, BF16, F32, 0, True),
    (2049, 9000, 40, BF16, BF16, 8, True), (20011, 70001, 16, F32, F16, 0, False), (300, 4, 4104, BF16, F32, 0, False),
])
def test_gradient(law, n, rows, dim, up, out, extra, accumulate):
    g = torch.Generator().manual_seed(n + dim)
    e, _ = _make(rows, dim, F32, scale=0.7, grad=out)
    before = e.grad.double().cpu() if accumulate else None
    tok = LAWS[law](n, rows, g).cuda()
    u = _wide(n, dim, extra, up)[:, :dim]
    u.copy_(torch.randn(n, dim, generator=g))
    e.backward(tok, u, accumulate=accumulate)
    e.sync()
    _check_grad(e, tok, u, before, 0.7, None, out)
    first = e.grad.clone()
    if not accumulate:
        e.backward(tok, u)
        e.sync()
        assert torch.equal(first.view(torch.uint8), e.grad.view(torch.uint8))   # the same bits


@pytest.mark.parametrize("n", [1, 20, 256, 257, 4000, 70000, 140000])
@pytest.mark.parametrize("rows,dim,shift", [(3, 1, 1), (50, 3, 1), (7, 24, 1), (1000, 8, 3), (33000, 1, 0), (4099, 20, 5), (2, 5000, 2),
                                            (900001, 2, 1), (3000001, 1, 0), (70001, 40, 0)])
@pytest.mark.parametrize("out", [F32, BF16])
def test_gradient_buffer_that_begins_anywhere(n, rows, dim, shift, out):
    """Every value of the buffer is written, none beside it; rows of one value, blocks of many rows."""
    g = torch.Generator().manual_seed(n)
    buf = torch.full((shift + rows * dim + 9,), 5.0, dtype=out, device="cuda")
    e = DenseEmbedding(rows, dim)
    e.set_table(torch.zeros(rows, dim, device="cuda"), grad=buf[shift:shift + rows * dim].view(rows, dim))
    tok = torch.randint(max(1, rows // 2), (n,), generator=g) * 2 % rows
    u = torch.randn(n, dim, generator=g)
    e.backward(tok.cuda(), u.cuda())
    e.sync()
    _check_grad(e, tok, u, None, 1.0, None, out)
    assert (buf[:shift] == 5.0).all() and (buf[shift + rows * dim:] == 5.0).all()


@pytest.mark.parametrize("n,rows,dim,pad", [(500, 40, 24, 3), (40000, 90, 8, 0), (3000, 1, 16, 0), (70, 33, 33, 32)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_padding_gets_no_gradient(n, rows, dim, pad, accumulate):
    g = torch.Generator().manual_seed(n)
    e, w = _make(rows, dim, F32, pad=pad, grad=F32)
    before = e.grad.double().cpu()
    tok = torch.randint(rows, (n,), generator=g, dtype=torch.int32)
    tok[torch.rand(n, generator=g) < 0.5] = pad
    u = torch.randn(n, dim, generator=g)
    u[tok == pad] = float("nan")                  # what lies at padded places is not read into a sum
    e.backward(tok.cuda(), u.cuda(), accumulate=accumulate)
    e.sync()
    _check_grad(e, tok, torch.nan_to_num(u), before if accumulate else None, 1.0, pad, F32)
    assert torch.equal(e.forward(tok.cuda()).cpu(), w[tok.long()])        # looked up like any row


def test_infinities_stay_in_their_row():
    e, _ = _make(50, 16, F32, grad=F32)
    tok = torch.arange(200, device="cuda") % 50
    u = torch.randn(200, 16, device="cuda")
    u[3, 5], u[7, 2] = float("inf"), float("nan")
    e.backward(tok, u)
    e.sync()
    bad = ~torch.isfinite(e.grad)
    assert bad.sum() == 2 and e.grad[3, 5] == float("inf") and torch.isnan(e.grad[7, 2])


def test_broadcast_upstream():
    e, _ = _make(20, 24, F32, grad=F32)
    tok = torch.randint(20, (700,), device="cuda")
    one = torch.randn(24, device="cuda")
    e.backward(tok, one.expand(700, 24))
    e.sync()
    _check_grad(e, tok, one.expand(700, 24), None, 1.0, None, F32)


@pytest.mark.parametrize("make", [lambda u: u.expand(5, 7, 24), lambda u: u.expand(35, 24)])
def test_expanded_upstream_of_any_shape(make):
    e, _ = _make(20, 24, F32, grad=F32)
    tok = torch.randint(20, (35,), device="cuda")
    up = make(torch.randn(24, device="cuda"))
    e.backward(tok.view(up.shape[:-1]), up)
    e.sync()
    _check_grad(e, tok, up.reshape(35, 24), None, 1.0, None, F32)


def test_a_captured_call_keeps_its_workspace():
    """Growing the workspace after a capture leaves the captured call's own in place."""
    e, _ = _make(300, 64, F32, grad=F32)
    tok, u = torch.randint(300, (3000,), device="cuda"), torch.randn(3000, 64, device="cuda")
    e.reserve(3000)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e.backward(tok, u)
    big, v = torch.randint(300, (50000,), device="cuda"), torch.randn(50000, 64, device="cuda")
    e.backward(big, v)
    _check_grad(e, big, v, None, 1.0, None, F32)
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    graph.replay()
    torch.cuda.synchronize()
    _check_grad(e, tok, u, None, 1.0, None, F32)
    e.sync()
    assert all((j == 255).all() for j in junk)


def test_results_allocated_on_the_given_stream():
    e, w = _make(64, 4096, F32)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(20):
        tok = torch.full((500,), k, device="cuda")
        torch.cuda.synchronize()
        out = e.forward(tok, stream=s if k % 2 else s.cuda_stream)
        s.synchronize()
        assert torch.equal(out[::250].cpu(), w[[k, k]])


def test_offsets_beyond_32_bits():
    rows, dim = 140001, 32768                       # 4.6e9 values
    w = torch.empty(rows, dim, dtype=BF16, device="cuda")
    e = DenseEmbedding(rows, dim, dtype=BF16)
    e.set_table(w, grad=torch.full_like(w, 5.0))
    tok = torch.tensor([rows - 1, 0, rows - 2, rows - 1], device="cuda")
    w[tok] = torch.randn(4, dim, device="cuda", dtype=BF16)
    assert torch.equal(e.forward(tok), w[tok])
    u = torch.randn(4, dim, device="cuda", dtype=BF16)
    e.backward(tok, u)
    e.sync()
    assert torch.equal(e.grad[rows - 1], (u[0].float() + u[3].float()).to(BF16))
    assert torch.equal(e.grad[rows - 2], u[2]) and torch.equal(e.grad[0], u[1])
    assert all(not e.grad[k:k + 10000].any() for k in range(1, rows - 2, 10000) if k + 10000 <= rows - 2)


def test_long_batch():
    """More upstream values than 2^32, each row far behind the last."""
    n, dim = 300001, 16384
    e, _ = _make(5, dim, BF16, grad=F32)
    tok = torch.arange(n, device="cuda") % 5
    u = torch.empty(n, dim, dtype=BF16, device="cuda").normal_()
    e.backward(tok, u)
    e.sync()
    k = 7 * 1024
    part = u[:, k:k + 32].double().cpu()
    want = torch.zeros(5, 32, dtype=torch.float64).index_add_(0, tok.cpu(), part)
    # 60001 terms: at most 60003 roundings of the sum of magnitudes, in whatever order
    size = torch.zeros(5, 32, dtype=torch.float64).index_add_(0, tok.cpu(), part.abs())
    assert ((e.grad[:, k:k + 32].double().cpu() - want).abs() <= 60003 * U * size).all()


@pytest.mark.parametrize("what", ["forward", "backward"])
@pytest.mark.parametrize("bad", [-1, 30, 2 ** 31 - 1, -2 ** 31, 2 ** 40])
@pytest.mark.parametrize("n", [10, 5000])
def test_tokens_outside_the_table(what, bad, n):
    e, w = _make(30, 8, F32, grad=F32)
    tok = torch.randint(30, (n,), dtype=torch.int64 if bad >= 2 ** 31 else torch.int32)
    ok = tok.clone().cuda()
    tok[n // 2] = bad
    u = torch.randn(n, 8, device="cuda")
    if what == "forward":
        e.forward(tok.cuda())
    else:
        e.backward(tok.cuda(), u)
    marked = torch.full((n, 8), 3.0, device="cuda")
    e.forward(ok, out=marked)                       # does nothing until the error is read
    with pytest.raises(abi.TTEmbError) as err:
        e.sync()
    assert err.value.code == abi.TT_ERR_INDEX_RANGE
    assert (marked == 3.0).all()
    assert abi.tt_emb_dense_last_error(e.handle) == abi.TT_ERR_INDEX_RANGE
    assert abi.tt_emb_dense_last_error(e.handle) == abi.TT_OK
    assert torch.equal(e.forward(ok).cpu(), w[ok.cpu().long()])
    e.backward(ok, u)
    e.sync()
    _check_grad(e, ok, u, None, 1.0, None, F32)


def test_refusals():
    e = DenseEmbedding(10, 4)
    tok = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(abi.TTEmbError) as err:
        e.forward(tok)                              # no table
    assert err.value.code == abi.TT_ERR_STATE
    w = torch.randn(10, 4, device="cuda")
    for bad, kind in ((w.cpu(), TypeError), (w.half(), TypeError), (w[:9], ValueError), (w.t().contiguous().t(), TypeError)):
        with pytest.raises(kind):
            e.set_table(bad)
    with pytest.raises(ValueError):
        e.set_table(w, grad=w[:, :3].contiguous())
    e.set_table(w, with_grad=False)
    with pytest.raises(abi.TTEmbError) as err:
        e.backward(tok, torch.zeros(3, 4, device="cuda"))   # no gradient buffer
    assert err.value.code == abi.TT_ERR_STATE
    e.set_table(w)
    for bad, kind in ((tok.cpu(), TypeError), (tok.float(), TypeError), (torch.zeros(6, dtype=torch.int64, device="cuda")[::2], ValueError)):
        with pytest.raises(kind):
            e.forward(bad)
    up = torch.zeros(3, 4, device="cuda")
    for bad, kind in ((up[:2], ValueError), (up.double(), TypeError), (up.cpu(), TypeError), (up.t().contiguous().t(), ValueError),
                      (torch.zeros(3, 2, 4, device="cuda")[:, 0].t().contiguous().t(), ValueError),
                      (torch.zeros(4, 3, device="cuda"), ValueError)):
        with pytest.raises(kind):
            e.backward(tok, bad)
    with pytest.raises(abi.TTEmbError) as err:      # rows of the output that overlap
        e.forward(tok, out=torch.zeros(1, 4, device="cuda").expand(3, 4))
    assert err.value.code == abi.TT_ERR_ARG
    fresh = DenseEmbedding(10, 4)
    fresh.set_table(w)
    with pytest.raises(abi.TTEmbError) as err:      # no workspace
        abi.tt_emb_dense_backward(fresh.handle, tok, up, 4)
    assert err.value.code == abi.TT_ERR_WORKSPACE
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(abi.TTEmbError) as err:
        abi.tt_emb_dense_set_workspace(fresh.handle, small, 1000)
    assert err.value.code == abi.TT_ERR_WORKSPACE
    fresh.reserve(3)
    with pytest.raises(abi.TTEmbError) as err:      # more tokens than reserved
        abi.tt_emb_dense_backward(fresh.handle, torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, 4, device="cuda"), 4)
    assert err.value.code == abi.TT_ERR_WORKSPACE
    assert abi.tt_emb_dense_last_error(fresh.handle) == abi.TT_ERR_WORKSPACE


@pytest.mark.parametrize("n", [37, 6000])
def test_captured_calls_replay_on_new_tokens(n):
    e, w = _make(500, 48, F32, grad=F32)
    tok, u = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.randn(n, 48, device="cuda")
    out = torch.empty(n, 48, device="cuda")
    s = torch.cuda.Stream()
    e.reserve(n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        e.forward(tok, out=out)
        e.backward(tok, u)
    for seed in (1, 2):
        new = torch.randint(500, (n,), generator=torch.Generator().manual_seed(seed))
        tok.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), w[new])
        _check_grad(e, new, u, None, 1.0, None, F32)
    e.sync()


def test_two_tables_on_two_streams():
    es = [_make(400, 32, F32, grad=F32, seed=k)[0] for k in range(2)]
    tok = [torch.randint(400, (9000,), device="cuda") for _ in es]
    up = [torch.randn(9000, 32, device="cuda") for _ in es]
    streams = [torch.cuda.Stream() for _ in es]
    torch.cuda.synchronize()
    for _ in range(5):
        for e, t, u, s in zip(es, tok, up, streams):
            e.reserve(9000)
            e.backward(t, u, stream=s)
    for e, t, u in zip(es, tok, up):
        e.sync()
        _check_grad(e, t, u, None, 1.0, None, F32)
