"""Calls large enough for the kernels that the size rules give to large batches, tables and lists.

Each test computes the rule that its size is to pass, with the card's own number of SMs, so that the size stays on
the wanted side of it.  Tolerances are those of test_gpu_dense.py and test_gpu_adamw.py, which derive them.
"""
import numpy as np
import pytest
import torch

from tensor_train_compressed_mixed_b200 import AdamW, DenseEmbedding, abi
from test_gpu_adamw import B1, B2, EPS, _check8, _check32, _fill, _snapshot, _tensors
from test_gpu_dense import U, _half_step, _least, _wide

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _up(a, b):
    return -(-a // b)


def _width(dim, a, b):
    """Values that one access moves, of rows that begin at multiples of 16 bytes if `dim` does."""
    most = 4 if a == b == F32 else 8
    return most if dim % most == 0 else 2 if dim % 2 == 0 else 1


def _tokens_a_unit(n, dim, table, out):
    """The lookup's units: tokens in one, and how many of them one step moves."""
    v = _width(dim, table, out)
    vectors = _up(dim, v)
    lanes = 1
    while lanes < vectors and lanes < 32:
        lanes *= 2
    slabs = _up(vectors, 32 if v > 2 else 64)
    k = 32 // lanes
    while k < 32 and _up(n, 2 * k) * slabs >= _sms() * 64:
        k *= 2
    return k, 32 // lanes, v


# ------------------------------------------------------------------ lookup
@pytest.mark.parametrize("n,dim,table,out,width,tokens,steps", [
    (4801, 4099, F32, F32, 1, 32, 32), (2500, 4099, BF16, F32, 1, 16, 16), (320007, 7, F16, BF16, 1, 32, 8), (400003, 1, F32, F32, 1, 32, 1),
    (9401, 4102, BF16, BF16, 2, 32, 32), (1300, 4102, F32, F16, 2, 4, 4), (320007, 6, F32, F32, 2, 32, 4), (50021, 514, F16, F16, 2, 16, 16),
    (18011, 2052, F32, F32, 4, 32, 32), (400009, 12, F32, F32, 4, 32, 4),
    (18011, 4104, BF16, BF16, 8, 32, 32), (9001, 4104, F32, BF16, 8, 16, 16), (320007, 24, F16, F32, 8, 32, 4),
])
def test_lookup_in_many_steps(n, dim, table, out, width, tokens, steps):
    k, rows, v = _tokens_a_unit(n, dim, table, out)
    assert (k, _up(k, rows), v) == (tokens, steps, width)
    g = torch.Generator(device="cuda").manual_seed(n)
    rows = 1009
    w = torch.randn(rows, dim, generator=g, device="cuda").to(table)
    e = DenseEmbedding(rows, dim, dtype=table, scale=3.7)
    e.set_table(w, with_grad=False)
    tok = torch.randint(rows, (n,), generator=g, device="cuda", dtype=torch.int32)
    extra = 0 if width > 2 else width                # keeps the width, and shows what is written between rows
    buf = _wide(n, dim, extra, out)
    e.forward(tok, out=buf[:, :dim])
    e.sync()
    assert (buf[:, dim:] == 7.0).all()
    step = max(1, (1 << 24) // dim)
    for i in range(0, n, step):
        want = w[tok[i:i + step].long()].double() * float(np.float32(3.7))
        tol = (_half_step(out) + U) * (1 + U) * want.abs() + _least(out)
        assert (buf[i:i + step, :dim].double() - want).abs().sub(tol).max() <= 0


@pytest.mark.parametrize("n,dim", [(4801, 4099), (18011, 2052)])
@pytest.mark.parametrize("where", [0, 17, -1])
def test_bad_token_in_many_steps(n, dim, where):
    e = DenseEmbedding(50, dim)
    w = torch.randn(50, dim, device="cuda")
    e.set_table(w, with_grad=False)
    assert _tokens_a_unit(n, dim, F32, F32)[0] == 32
    tok = torch.randint(50, (n,), device="cuda")
    ok = tok.clone()
    tok[where] = 50
    buf = torch.full((n + 1, dim), 7.0, device="cuda")
    e.forward(tok, out=buf[:n])
    with pytest.raises(abi.TTEmbError) as err:
        e.sync()
    assert err.value.code == abi.TT_ERR_INDEX_RANGE
    assert (buf[n] == 7.0).all() and (buf[where if where >= 0 else n - 1] == 7.0).all()    # a row that is not there is not written
    e.forward(ok, out=buf[:n])
    e.sync()
    assert torch.equal(buf[:n], w[ok])


# ------------------------------------------------------------------ gradient
def _check_gradient(e, tok, up, before, scale, pad, out):
    """e.grad against sums in 64 bits on the device, some columns at a time."""
    rows, dim = e.num_rows, e.dim
    t = tok.long()
    keep = torch.ones_like(t, dtype=torch.bool) if pad is None else t != pad
    t, s = t[keep], float(np.float32(scale))
    k = torch.bincount(t, minlength=rows).double()[:, None]
    for c in range(0, dim, 512):
        u = up[:, c:c + 512][keep].double()
        want = torch.zeros(rows, u.shape[1], dtype=torch.float64, device="cuda").index_add_(0, t, u) * s
        size = torch.zeros_like(want).index_add_(0, t, u.abs()) * abs(s)
        if before is not None:
            b = before[:, c:c + 512].double()
            want, size = want + b, size + b.abs()
        tol = (k + 2) * U * 1.01 * size + _half_step(out) * (1 + 1e-3) * want.abs() + _least(out)
        got = e.grad[:, c:c + 512].double()
        assert (got - want).abs().sub(tol).max() <= 0
        if before is None:
            assert not got[k[:, 0] == 0].any()


def _tile(n, dim, v):
    slabs = _up(dim, 32 * (v if v > 2 else 8 if v == 2 else 4))
    units, want = _up(n, 32) * slabs, _sms() * 24
    return (32 if units <= want else 32 * min(8, units // want)), slabs


@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("law", ["uniform", "zipf", "runs"])
@pytest.mark.parametrize("n,rows,dim,up,out,width,tile,extra", [
    (20011, 3001, 2056, BF16, F32, 8, 32, 8), (20011, 3001, 1030, BF16, BF16, 2, 32, 2), (20011, 3001, 515, F16, F32, 1, 32, 3),
    (20011, 3001, 1028, F32, F32, 4, 32, 0), (40009, 9001, 2056, F32, F16, 8, 96, 0), (65537, 500, 1030, F32, BF16, 2, 64, 0),
    (140011, 2003, 1028, F32, F32, 4, 256, 4), (140011, 20011, 515, BF16, BF16, 1, 192, 0),
])
def test_gradient_of_many_units(accumulate, law, n, rows, dim, up, out, width, tile, extra):
    got, slabs = _tile(n, dim, width)
    assert _width(dim, up, out) == width and got == tile
    assert _up(n, tile) * slabs > _sms() * 16        # fewer units take eight rows at a time
    g = torch.Generator(device="cuda").manual_seed(n + dim)
    if law == "uniform":
        tok = torch.randint(rows, (n,), generator=g, device="cuda")
    elif law == "zipf":
        r = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
        tok = (torch.exp(r * float(np.log(rows))) - 1).long().clamp_(0, rows - 1)
    else:
        tok = (torch.arange(n, device="cuda") // tile) % rows      # runs that end where tiles do, at first
    pad = rows // 3
    e = DenseEmbedding(rows, dim, scale=0.7, padding_idx=pad)
    e.set_table(torch.zeros(rows, dim, device="cuda"), grad=torch.randn(rows, dim, generator=g, device="cuda").to(out))
    before = e.grad.clone() if accumulate else None
    u = _wide(n, dim, extra, up)[:, :dim]
    u.copy_(torch.randn(n, dim, generator=g, device="cuda"))
    e.backward(tok, u, accumulate=accumulate)
    e.sync()
    _check_gradient(e, tok, u, before, 0.7, pad, out)


@pytest.mark.parametrize("n", [4, 300])
def test_clearing_beyond_32_bits(n):
    """Rows whose values lie behind the first 2^32, all of them, where one launch clears and where sums and joins do."""
    rows, dim = 140001, 32768
    e = DenseEmbedding(rows, dim, dtype=BF16)
    e.set_table(torch.zeros(rows, dim, dtype=BF16, device="cuda"), grad=torch.full((rows, dim), 5.0, dtype=BF16, device="cuda"))
    tok = torch.randint(rows, (n,), generator=torch.Generator().manual_seed(n))
    tok[:4] = torch.tensor([rows - 1, 0, rows - 2, rows - 1])
    tok = tok.cuda()
    u = torch.randn(n, dim, device="cuda", dtype=BF16)
    e.backward(tok, u)
    e.sync()
    named = torch.zeros(rows, dtype=torch.bool, device="cuda")
    named[tok] = True
    for k in range(0, rows, 10000):
        part = e.grad[k:k + 10000]
        assert not part[~named[k:k + 10000]].any()
    for r in (0, rows - 2, rows - 1):
        one = u[tok == r].float()
        assert ((e.grad[r].float() - one.sum(0)).abs() <= (2.0 ** -8 + 4 * U) * one.abs().sum(0)).all()


# ------------------------------------------------------------------ AdamW
def test_step_32_in_many_turns():
    """More tiles than blocks of threads, so that blocks take tile after tile, of several tensors."""
    for ptype, gtype, shift in ((F32, F32, 0), (BF16, BF16, 0), (F16, F32, 1)):
        sizes = [900003, 1, 700001, 255]
        assert sum(_up(n, 2048) for n in sizes) > 2 * _sms() * 2
        ps, gs = _tensors(sizes, ptype, gtype, shift=shift)
        o = AdamW(ps, gs, betas=(B1, B2), eps=EPS, weight_decay=0.1)
        _fill(o)
        o.steps.fill_(5)
        before = [[x.clone() for x in (p, g, o.m[a:a + p.numel()], o.v[a:a + p.numel()])] for p, g, a in zip(ps, gs, o.offsets)]
        o.step(0.01)
        assert int(o.steps) == 6
        for (p0, g0, m0, v0), p, a in zip(before, ps, o.offsets):
            n = p.numel()
            _check32(p0, g0, m0, v0, p, o.m[a:a + n], o.v[a:a + n], 6, float(np.float32(0.01)), 0.1)


@pytest.mark.parametrize("ptype,gtype,shift,sizes,each", [
    (BF16, BF16, 0, [5100003, 300, 1], 9), (F32, F32, 0, [9300007, 70001], 16), (BF16, F32, 0, [257, 9300007], 16),
    (F16, BF16, 1, [12000001, 255, 40001], 16),
])
def test_steps_8_of_many_blocks_a_warp(ptype, gtype, shift, sizes, each):
    """Warps that take several blocks in a row, fetched ahead, each with its own scale and random words, and (the last
    list) blocks of threads that take a second tile."""
    blocks = [_up(n, 256) for n in sizes]
    per = 1
    while per < 16 and sum(_up(b, per * 8) for b in blocks) > _sms() * 2:
        per += 1
    assert per == each
    assert (sum(_up(b, per * 8) for b in blocks) > _sms() * 2) == (max(sizes) > 11 << 20)
    ps, gs = _tensors(sizes, ptype, gtype, shift=shift)
    # blocks of unlike magnitudes, so that a scale or a stage of another block shows
    for g in gs:
        k = torch.arange(g.numel(), device="cuda") // 256
        g.mul_(torch.exp2((k * 7 % 11 - 8).float()).to(g.dtype))
    seed = 77
    o = AdamW(ps, gs, betas=(B1, B2), eps=EPS, weight_decay=0.1, state_bits=8, seed=seed)
    for t in (1, 2):
        before = _snapshot(o)
        o.step(0.01)
        _check8(o, before, t, float(np.float32(0.01)), 0.1, seed)
        for g in gs:
            g.mul_(-0.7)
