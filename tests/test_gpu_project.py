"""The table as a matrix (DenseEmbedding.project and .project_backward) against the formulas in 64 bits.

Tolerances count roundings.  A sum of k products held in fp32 is off by at most k + 2 steps of 2^-23 of the sum of
magnitudes (a step, not half: tensor cores cut their sums' last bits off); fp32 operands as three bf16 terms leave
2^-22 of a product out at most.  An activation stretches that by its slope, at most 1.13, and is itself off by 16 steps of fp32; where the result has 16 bits by 2^-15 of its value (a fit
within 5.2e-6, and an exponent of 2 below 2^7 rounded twice to 24 bits: 2 * 2^7 * 2^-24 * ln 2 = 1.1e-5).
A result is rounded once, by half a step of its type.  Where a 16-bit result's products take dz in 16 bits, each term
is off by half a step of that type.
"""
import math
import os
import subprocess

import pytest
import torch

from tensor_train_compressed_mixed_b200 import AdamW, DenseEmbedding, GradNorm, TTEmbError, abi

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
STEP = 2.0 ** -23


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _least(dtype):
    return torch.finfo(dtype).smallest_normal * _half_step(dtype)


def _act64(act, z, cap):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "silu":
        return z * torch.sigmoid(z)
    return cap * torch.tanh(z / cap) if act == "softcap" else z


def _wide(n, width, extra, dtype, fill=7.0):
    return torch.full((n, width + extra), fill, dtype=dtype, device="cuda")


def _randn(g, *shape, dtype=F32, by=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * by).to(dtype)


def _table(rows, dim, kind, g, grad=None, pad=None):
    w = _randn(g, rows, dim, dtype=kind, by=1 / math.sqrt(dim))
    e = DenseEmbedding(rows, dim, dtype=kind, scale=5.0, padding_idx=pad)
    e.set_table(w, grad=grad, with_grad=False)
    return e, w


def _sum_tol(a, b, k):
    """Bound of |computed - exact| of a @ b over k terms, both in 64 bits."""
    return (a.abs() @ b.abs()) * ((k + 2) * STEP + 2.0 ** -22)


def _inside(got, want, tol):
    bad = ((got.double() - want).abs() > tol) | ~torch.isfinite(got.double())
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(((got.double() - want).abs() / tol.clamp(min=1e-300)).max()))


# n, rows, dim, table, out, activation, bias, residual, pre, extra
FORWARD = [
    (1, 1, 1, F32, F32, None, True, True, True, 0), (1, 1, 1, BF16, BF16, "gelu", True, False, True, 0),
    (1, 130, 64, F16, F32, "silu", True, True, True, 0), (3, 5, 8, BF16, BF16, "relu", False, True, False, 3),
    (2, 300, 4097, F32, F32, "softcap", True, False, False, 0), (16, 128, 64, BF16, F32, None, False, False, False, 0),
    (17, 127, 72, F16, F16, "gelu", True, True, True, 8), (33, 257, 129, BF16, BF16, "silu", True, True, True, 1),
    (64, 1000, 512, BF16, BF16, None, True, False, False, 0), (65, 1000, 520, F16, F16, "softcap", False, True, False, 0),
    (129, 385, 1000, BF16, F32, "gelu", True, True, True, 0), (257, 513, 256, F32, F32, "gelu", True, True, True, 5),
    (300, 70, 2048, F32, BF16, None, False, False, True, 0), (512, 640, 192, BF16, F16, "relu", True, True, False, 8),
    (1000, 2100, 100, F16, F16, "silu", True, True, True, 4), (5, 40000, 64, BF16, BF16, None, True, False, False, 0),
    (700, 3, 900, BF16, BF16, None, True, True, True, 1), (2050, 1030, 520, BF16, BF16, "gelu", True, True, False, 0),
    (8, 5000, 8192, BF16, F32, "softcap", False, False, False, 0), (100, 50, 20000, F16, F32, None, True, False, False, 0),
    (3001, 9000, 200, BF16, BF16, "gelu", True, True, True, 0), (3000, 9002, 136, F16, F32, "silu", True, True, False, 2),
    (4100, 4360, 72, F32, F32, None, False, False, False, 0), (32, 30000, 97, F32, F32, "gelu", True, True, True, 3), (7, 20011, 515, BF16, BF16, None, True, True, False, 1), (4, 20, 30000, BF16, BF16, "gelu", True, True, True, 1), (31, 70000, 128, F16, F16, "relu", True, True, True, 0),
]


@pytest.mark.parametrize("n,rows,dim,kind,out,act,bias,residual,pre,extra", FORWARD)
def test_project(n, rows, dim, kind, out, act, bias, residual, pre, extra):
    g = torch.Generator(device="cuda").manual_seed(n * 7 + rows + dim)
    e, w = _table(rows, dim, kind, g)
    x = _wide(n, dim, extra, kind)
    x[:, :dim] = _randn(g, n, dim, dtype=kind)
    x = x[:, :dim]
    b = _randn(g, rows, dtype=out) if bias else None
    res = _randn(g, n, rows + extra, dtype=BF16)[:, :rows] if residual else None
    z_buf, y_buf = _wide(n, rows, extra, F32), _wide(n, rows, extra, out)
    cap = 2.5 if act == "softcap" else None
    got = e.project(x, bias=b, activation=act, cap=cap, residual=res, out=y_buf[:, :rows], pre=z_buf[:, :rows] if pre else None)
    e.sync()
    z = x.double() @ w.double().t()
    tol = _sum_tol(x.double(), w.double().t(), dim)
    if bias:
        z = z + b.double()
        tol = tol + 2 * STEP * z.abs()
    if pre:
        _inside(z_buf[:, :rows], z, tol + STEP * z.abs())
        assert (z_buf[:, rows:] == 7).all()
    want = _act64(act, z, cap)
    tol = 1.13 * tol + (16 * STEP if out == F32 else 2.0 ** -15) * (want.abs() + 2.0 ** -100)
    if residual:
        want = want + res.double()
        tol = tol + STEP * want.abs()
    _inside(got, want, tol + _half_step(out) * (want.abs() + tol) + _least(out))
    assert (y_buf[:, rows:] == 7).all()


# n, rows, dim, table, grad_out, grad_x, grad, activation, bias, accumulate, extra, padding row
BACKWARD = [
    (1, 1, 1, F32, F32, F32, F32, None, True, True, 0, None), (1, 1, 1, BF16, BF16, BF16, BF16, "gelu", True, False, 0, None),
    (1, 200, 70, F32, F32, F32, F32, "silu", True, True, 0, 5), (3, 5, 8, BF16, BF16, BF16, F32, "relu", True, False, 3, 0),
    (64, 128, 64, BF16, BF16, BF16, BF16, None, True, False, 0, 127), (200, 1000, 512, BF16, BF16, BF16, BF16, "silu", True, True, 0, None),
    (65, 129, 257, F32, F32, F32, F32, "softcap", True, True, 5, 1), (129, 300, 72, F16, F16, F16, F32, "gelu", True, False, 8, None),
    (257, 500, 136, F16, F32, F16, F16, None, True, False, 0, 3), (100, 2000, 96, BF16, F32, BF16, BF16, "silu", False, False, 0, None),
    (300, 77, 1000, BF16, BF16, F32, F32, "gelu", True, True, 1, None), (1000, 2100, 130, F16, F16, F16, F16, "silu", True, False, 0, None),
    (2050, 1030, 128, BF16, BF16, BF16, F32, None, True, True, 0, 1029), (9, 30000, 64, BF16, BF16, BF16, BF16, None, False, False, 0, None),
    (4000, 40, 24, BF16, BF16, BF16, BF16, "gelu", True, False, 0, None), (500, 257, 520, F32, BF16, BF16, BF16, "gelu", True, False, 0, None),
    (4100, 3000, 1288, BF16, BF16, BF16, BF16, "silu", True, True, 0, 17), (5000, 2600, 1100, F16, F16, F32, F32, None, False, False, 4, None),
    (2, 40000, 100, BF16, BF16, BF16, BF16, "relu", True, False, 0, None), (20, 50000, 33, F32, F32, F32, F32, None, True, True, 3, 9),
    (5, 30011, 64, F16, F16, F32, F16, "gelu", True, False, 1, None), (30, 9000, 2000, F32, F32, F32, F32, None, True, False, 0, None), (513, 640, 264, F16, F16, F32, F32, None, False, False, 0, None),
]


def _is_narrow(kind, up, result, act):
    """Whether a result's products take dz in the table's 16 bits, and whether that rounds it."""
    if kind == F32 or (kind == F16 and up == F32):
        return False
    return result != F32 and not (act is None and up == kind)


@pytest.mark.parametrize("n,rows,dim,kind,up,gx,gw,act,bias,accumulate,extra,pad", BACKWARD)
def test_project_backward(n, rows, dim, kind, up, gx, gw, act, bias, accumulate, extra, pad):
    g = torch.Generator(device="cuda").manual_seed(n * 5 + rows + dim)
    start = _randn(g, rows, dim, dtype=gw)
    e, w = _table(rows, dim, kind, g, grad=start.clone(), pad=pad)
    x = _randn(g, n, dim + extra, dtype=kind)[:, :dim]
    dy = _randn(g, n, rows + extra, dtype=up)[:, :rows]
    z = _randn(g, n, rows + extra, dtype=up)[:, :rows] if act else None
    cap = 2.5 if act == "softcap" else None
    gb = _randn(g, rows) if bias else None
    gb0 = gb.clone() if bias else None
    gx_buf = _wide(n, dim, extra, gx)
    got = e.project_backward(x, dy, pre=z, activation=act, cap=cap, accumulate=accumulate, grad_x=gx_buf[:, :dim], grad_bias=gb)
    e.sync()
    d = dy.double()
    off = torch.zeros_like(d)
    if act:
        zz = z.double().requires_grad_()
        d, = torch.autograd.grad(_act64(act, zz, cap), zz, d)
        off = 32 * STEP * dy.double().abs()       # the slope in fp32
    def rounded(result):
        narrow = _is_narrow(kind, up, result, act)
        return off + _half_step(kind) * (d.abs() + off) + _least(kind) if narrow else off + 2.0 ** -22 * d.abs()
    want = d @ w.double()
    tol = _sum_tol(d, w.double(), rows) + rounded(gx) @ w.double().abs()
    _inside(got, want, tol + _half_step(gx) * (want.abs() + tol) + _least(gx))
    assert (gx_buf[:, dim:] == 7).all()
    dt = d.t().clone()
    rt = rounded(gw).t().clone()
    if pad is not None:
        dt[pad] = 0
        rt[pad] = 0
    want = dt @ x.double()
    tol = _sum_tol(dt, x.double(), n) + rt @ x.double().abs()
    if accumulate:
        want = want + start.double()
        tol = tol + STEP * want.abs()
    _inside(e.grad, want, tol + _half_step(gw) * (want.abs() + tol) + _least(gw))
    if pad is not None:
        assert torch.equal(e.grad[pad], start[pad] if accumulate else torch.zeros_like(start[pad]))
    if bias:
        want = d.sum(0) + (gb0.double() if accumulate else 0)
        _inside(gb, want, d.abs().sum(0) * (n + 4) * STEP + off.sum(0) + STEP * want.abs())


@pytest.mark.parametrize("act", ["gelu", "silu", "softcap", "relu"])
@pytest.mark.parametrize("kind", [F32, BF16])
def test_gradients_are_the_differences(act, kind):
    """<dy, (f(x + h dx) - f(x - h dx)) / 2 h> against <grad_x, dx> and the like for the table and the bias, all
    differences by the formula in 64 bits.  The third derivative leaves h^2, the gradients' own roundings the rest."""
    n, rows, dim, cap = 20, 150, 90, 2.5 if act == "softcap" else None
    g = torch.Generator(device="cuda").manual_seed(3)
    e, w = _table(rows, dim, kind, g, grad=torch.zeros(rows, dim, device="cuda"))
    x, b, dy = _randn(g, n, dim, dtype=kind), _randn(g, rows), _randn(g, n, rows, dtype=kind)
    pre = torch.empty(n, rows, device="cuda")
    e.project(x, bias=b, activation=act, cap=cap, pre=pre)
    gb, gx = torch.empty_like(b), torch.empty(n, dim, device="cuda")
    e.project_backward(x, dy, pre=pre, activation=act, cap=cap, grad_x=gx, grad_bias=gb)
    e.sync()
    f = lambda x, w, b: (dy.double() * _act64(act, x @ w.t() + b, cap)).sum()  # noqa: E731
    at = [x.double(), w.double(), b.double()]
    for i, got in enumerate((gx, e.grad, gb)):
        step = _randn(g, *at[i].shape).double()
        h = 1e-5
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * step, at[i] - h * step
        want = (f(*up) - f(*down)) / (2 * h)
        size = (got.double().abs() * step.abs()).sum()
        assert abs(float((got.double() * step).sum() - want)) <= 1e-5 * float(size), (act, i)   # relu's kinks lie within h: 1e-5 of them


def test_broadcast_rows_and_shapes():
    g = torch.Generator(device="cuda").manual_seed(4)
    for kind, n, rows, dim in ((BF16, 40, 300, 128), (F32, 33, 65, 40)):
        e, w = _table(rows, dim, kind, g, grad=torch.zeros(rows, dim, device="cuda"))
        x = _randn(g, 1, dim, dtype=kind).expand(n, dim)                      # one row for all
        res = _randn(g, 1, rows).expand(n, rows)
        got = e.project(x, residual=res, out_dtype=F32)
        want = x.double() @ w.double().t() + res.double()
        _inside(got, want, _sum_tol(x.double(), w.double().t(), dim) + 2 * STEP * want.abs())
        dy = torch.ones(1, 1, dtype=kind, device="cuda").expand(n, rows)      # of a sum over all
        if kind == BF16:
            dy = _randn(g, 1, rows, dtype=kind).expand(n, rows)
        else:
            dy = dy.contiguous()
        gx = e.project_backward(x, dy, grad_x=torch.empty(n, dim, device="cuda"))
        _inside(gx, dy.double() @ w.double(), _sum_tol(dy.double(), w.double(), rows))
        _inside(e.grad, dy.double().t() @ x.double(), _sum_tol(dy.double().t(), x.double(), n))
        three = _randn(g, 2, 3, dim, dtype=kind)
        assert e.project(three).shape == (2, 3, rows)
        assert e.project_backward(three, _randn(g, 2, 3, rows, dtype=kind)).shape == (2, 3, dim)
        e.sync()


def test_empty_calls():
    e, w = _table(10, 6, F32, torch.Generator(device="cuda").manual_seed(1), grad=torch.ones(10, 6, device="cuda"))
    none = torch.empty(0, 6, device="cuda")
    assert e.project(none).shape == (0, 10)
    gb = torch.ones(10, device="cuda")
    assert e.project_backward(none, torch.empty(0, 10, device="cuda"), accumulate=True, grad_bias=gb).shape == (0, 6)
    assert (e.grad == 1).all() and (gb == 1).all()
    e.project_backward(none, torch.empty(0, 10, device="cuda"), grad_bias=gb)
    e.sync()
    assert (e.grad == 0).all() and (gb == 0).all()


def test_residual_in_place_and_parts_of_one_buffer():
    g = torch.Generator(device="cuda").manual_seed(5)
    for kind, n, rows, dim in ((BF16, 70, 256, 192), (F32, 20, 33, 17)):
        e, w = _table(rows, dim, kind, g)
        wide = _randn(g, n, dim + rows, dtype=kind)
        x, out = wide[:, :dim], wide[:, dim:]
        want = x.double() @ w.double().t() + out.double()
        tol = _sum_tol(x.double(), w.double().t(), dim) + STEP * want.abs()
        keep = x.clone()
        assert e.project(x, residual=out, out=out) is out
        e.sync()
        _inside(out, want, tol + _half_step(kind) * (want.abs() + tol))
        assert torch.equal(x, keep)
        with pytest.raises(TTEmbError):
            e.project(x, residual=out, out=wide[:, dim - 1:-1])


@pytest.mark.parametrize("kind", [F32, BF16, F16])
def test_infinities_and_nans_stay_in_their_rows(kind):
    """A row of x touches its own row of the result alone, whatever it holds; rows of the table their columns."""
    g = torch.Generator(device="cuda").manual_seed(6)
    n, rows, dim = 40, 300, 136
    e, w = _table(rows, dim, kind, g, grad=torch.zeros(rows, dim, device="cuda"))
    x = _randn(g, n, dim, dtype=kind)
    clean = e.project(x, out_dtype=F32).clone()
    x[3, 5], x[n - 1, dim - 1], w[7, 0], w[rows - 1, 100] = math.inf, math.nan, math.nan, -math.inf
    got = e.project(x, out_dtype=F32)
    e.sync()
    bad_r, bad_c = torch.zeros(n, dtype=torch.bool, device="cuda"), torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad_r[[3, n - 1]] = True
    bad_c[[7, rows - 1]] = True
    hit = bad_r[:, None] | bad_c[None, :]
    assert torch.equal(got[~hit], clean[~hit])
    assert not torch.isfinite(got[hit]).any()


def test_same_bits_every_time_and_on_another_stream():
    g = torch.Generator(device="cuda").manual_seed(7)
    for kind, n, rows, dim in ((BF16, 300, 2000, 512), (F32, 130, 700, 260), (BF16, 8, 700, 4096)):
        e, w = _table(rows, dim, kind, g, grad=torch.zeros(rows, dim, device="cuda"))
        x, dy, pre = _randn(g, n, dim, dtype=kind), _randn(g, n, rows, dtype=kind), _randn(g, n, rows, dtype=kind)
        gb = torch.empty(rows, device="cuda")

        def once(stream=None):
            y = e.project(x, activation="gelu", stream=stream)
            gx = e.project_backward(x, dy, pre=pre, activation="gelu", grad_bias=gb, stream=stream)
            if stream is not None:
                stream.synchronize()
            return [y.clone(), gx.clone(), e.grad.clone(), gb.clone()]
        first = once()
        torch.cuda.synchronize()
        for again in (once(), once(torch.cuda.Stream())):
            assert all(torch.equal(a, b) for a, b in zip(first, again))
        e.sync()


def test_captured_and_replayed_beside_eager_calls():
    g = torch.Generator(device="cuda").manual_seed(8)
    n, rows, dim = 96, 520, 200
    for kind in (BF16, F32):
        e, w = _table(rows, dim, kind, g, grad=torch.zeros(rows, dim, device="cuda"))
        x, dy, pre = _randn(g, n, dim, dtype=kind), _randn(g, n, rows, dtype=kind), torch.empty(n, rows, device="cuda")
        y, gx, gb = torch.empty(n, rows, dtype=kind, device="cuda"), torch.empty(n, dim, dtype=kind, device="cuda"), torch.empty(rows, device="cuda")

        def call():
            e.project(x, activation="silu", out=y, pre=pre)
            e.project_backward(x, dy, pre=pre, activation="silu", grad_x=gx, grad_bias=gb)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        x.copy_(_randn(g, n, dim, dtype=kind))
        bigger = _randn(g, 4 * n, dim, dtype=kind)
        e.project(bigger)                                   # another workspace for eager calls
        e.project_backward(bigger, _randn(g, 4 * n, rows, dtype=kind), pre=_randn(g, 4 * n, rows), activation="gelu")
        call()
        want = [t.clone() for t in (y, pre, gx, gb, e.grad)]
        for t in (y, pre, gx, gb, e.grad):
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, pre, gx, gb, e.grad)))
        e.sync()


def test_a_pending_device_error_stops_the_calls():
    g = torch.Generator(device="cuda").manual_seed(9)
    for kind, n, rows, dim in ((BF16, 64, 256, 256), (F32, 64, 300, 70), (BF16, 2, 700, 4096)):
        e, w = _table(rows, dim, kind, g, grad=torch.full((rows, dim), 5.0, device="cuda"))
        x, dy = _randn(g, n, dim, dtype=kind), _randn(g, n, rows, dtype=kind)
        out, gx, gb = torch.full((n, rows), 5.0, device="cuda"), torch.full((n, dim), 5.0, device="cuda"), torch.full((rows,), 5.0, device="cuda")
        e.forward(torch.tensor([rows], device="cuda"))
        e.project(x, out=out, activation="relu")
        e.project_backward(x, dy, pre=dy, activation="relu", grad_x=gx, grad_bias=gb)
        with pytest.raises(TTEmbError) as err:
            e.sync()
        assert err.value.code == abi.TT_ERR_INDEX_RANGE
        assert all((t == 5).all() for t in (out, gx, gb, e.grad))
        e.project(x, out=out)
        e.sync()
        assert not (out == 5).all()


def test_refusals():
    g = torch.Generator(device="cuda").manual_seed(10)
    e, w = _table(10, 6, BF16, g)
    x, dy = _randn(g, 4, 6, dtype=BF16), _randn(g, 4, 10, dtype=BF16)
    for bad in (x.float(), x.cpu()):
        with pytest.raises(TypeError):
            e.project(bad)
    for bad in (x[:, :5], x.t().contiguous(), x[0, 0]):
        with pytest.raises(ValueError):
            e.project(bad)
    with pytest.raises(ValueError):
        e.project(x, bias=torch.zeros(9, device="cuda"))
    with pytest.raises(ValueError):
        e.project(x, residual=torch.zeros(4, 9, device="cuda"))
    with pytest.raises(TypeError):
        e.project(x, out=torch.zeros(4, 10, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError):
        e.project(x, activation="gelu", cap=1.0)
    with pytest.raises(TTEmbError) as err:
        e.project_backward(x, dy)                     # no gradient buffer
    assert err.value.code == abi.TT_ERR_STATE
    assert e.project_backward(None, dy, table_grad=False).shape == (4, 6)
    with pytest.raises(ValueError):
        e.project_backward(x, dy[:, :9])
    with pytest.raises(ValueError):
        e.project_backward(x, dy, activation="gelu", table_grad=False)
    with pytest.raises(TTEmbError):
        e.project(x, out=dy, residual=dy.flip(0).flip(0)[:, :], pre=dy)


def test_a_training_run_of_a_tied_table():
    """Lookup, head and its gradients, the lookup's gradient added, clipping and the AdamW step, as they are used
    together, against the same in 64 bits from the same bf16 weights; the second half by SGD's clipping in place."""
    g = torch.Generator(device="cuda").manual_seed(11)
    rows, dim, n = 500, 64, 200
    grad = torch.zeros(rows, dim, device="cuda")
    e, w = _table(rows, dim, BF16, g, grad=grad)
    e.close()
    e = DenseEmbedding(rows, dim, dtype=BF16, scale=8.0)
    w0 = w.clone()
    e.set_table(w, grad=grad)
    bias, gb = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    opt = AdamW([w, bias], [grad, gb], weight_decay=0.0)
    ids = torch.randint(rows, (n,), generator=g, device="cuda")
    to = torch.randint(rows, (n,), generator=g, device="cuda")
    h = e.forward(ids)
    logits = e.project(h, bias=bias, out_dtype=F32)
    p = torch.softmax(logits, 1)
    p[torch.arange(n), to] -= 1
    dlogits = (p / n).to(BF16)
    dh = e.project_backward(h, dlogits, grad_bias=gb)
    e.backward(ids, dh, accumulate=True)
    norm = opt.step(1e-2, max_norm=0.01).clone()
    e.sync()
    W, H, D = w0.double(), h.double(), dlogits.double()
    want = D.t() @ H
    want.index_add_(0, ids, 8.0 * dh.double())
    tol = D.abs().t() @ H.abs() * (n * STEP) + STEP * n * want.abs().max()
    _inside(grad, want, tol + 1e-6)
    total = torch.sqrt(grad.double().square().sum() + gb.double().square().sum())
    assert abs(float(norm) - float(total)) <= 4 * STEP * float(total) and float(total) > 0.01
    by = 0.01 / total
    step = (grad.double() * by) / ((grad.double() * by).abs() + 1e-8)       # the first step's quotient
    _inside(w, W - 1e-2 * step, _half_step(BF16) * (W.abs() + 0.02) + 1e-2 * 1e-4)
    clip = GradNorm([grad, gb])
    assert abs(float(clip.clip(0.5 * float(total))) - float(total)) <= 4 * STEP * float(total)
    assert abs(float(clip.norm()) - 0.5 * float(total)) <= 8 * STEP * float(total)


@pytest.mark.parametrize("n,rows,dim", [(33000, 66000, 8), (3, 2 ** 21 + 5, 1032)])
def test_offsets_past_32_bits(n, rows, dim):
    """Results, or the table and its gradient, of more than 2^31 values: the last rows and columns."""
    g = torch.Generator(device="cuda").manual_seed(12)
    w = torch.zeros(rows, dim, dtype=BF16, device="cuda")
    grad = torch.zeros(rows, dim, dtype=BF16, device="cuda")
    e = DenseEmbedding(rows, dim, dtype=BF16)
    e.set_table(w, grad=grad)
    w[-300:] = _randn(g, 300, dim, dtype=BF16)
    x = _randn(g, n, dim, dtype=BF16)
    y = e.project(x)
    want = x[-3:].double() @ w[-300:].double().t()
    tol = _sum_tol(x[-3:].double(), w[-300:].double().t(), dim)
    _inside(y[-3:, -300:], want, tol + _half_step(BF16) * (want.abs() + tol) + _least(BF16))
    assert not y[-3:, :-300].any() and not y[:3, :-300].any()
    y.zero_()
    y[-3:, -300:] = _randn(g, 3, 300, dtype=BF16)
    gx = e.project_backward(x, y, grad_x=torch.empty(n, dim, device="cuda"))
    e.sync()
    d = y[-3:, -300:].double()
    _inside(gx[-3:], d @ w[-300:].double(), _sum_tol(d, w[-300:].double(), rows if rows < 10 ** 5 else 300 * 64))
    want = d.t() @ x[-3:].double()
    tol = _sum_tol(d.t(), x[-3:].double(), n)
    _inside(grad[-300:], want, tol + _half_step(BF16) * (want.abs() + tol) + _least(BF16))
    assert not grad[:-300].any()


NO_CLUSTERS = """
import ctypes
import torch
from tensor_train_compressed_mixed_b200 import DenseEmbedding, GradNorm
fake = ctypes.CDLL(None)
g = torch.Generator(device="cuda").manual_seed(1)
rand = lambda *s, t=torch.float32: torch.randn(*s, generator=g, device="cuda").to(t)
for kind, n, rows, dim in ((torch.bfloat16, 3000, 9000, 192), (torch.bfloat16, 9, 700, 4096), (torch.float32, 200, 500, 1000)):
    w, x, dy = rand(rows, dim, t=kind), rand(n, dim, t=kind), rand(n, rows, t=kind)
    got = []
    for none_fits in (1, 0):
        fake.fake_no_clusters(none_fits)
        before = fake.fake_cluster_launches()
        e = DenseEmbedding(rows, dim, dtype=kind)
        e.set_table(w, grad=torch.empty(rows, dim, device="cuda"))
        y = e.project(x, out_dtype=torch.float32)
        gx = e.project_backward(x, dy, grad_x=torch.empty(n, dim, device="cuda"))
        norm = GradNorm([e.grad])
        size = norm.clip(1.0).clone()
        short = GradNorm([rand(100)])
        short.clip(1.0)
        e.sync()
        assert (fake.fake_cluster_launches() > before) == (not none_fits)
        got.append((y, gx, e.grad, size))
    for a, b in zip(*got):
        assert (a - b).abs().max() <= 1e-4 * b.abs().max()
"""


def test_a_device_without_clusters(tmp_path):
    """Where no cluster of blocks fits the device, single blocks take the tiles and two launches clip."""
    from test_gpu_fake_runtime import _run
    so = tmp_path / "libfake.so"
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run(["gcc", "-O1", "-fPIC", "-shared", "-I/usr/local/cuda/include", os.path.join(here, "fake_cudart.c"), "-o", str(so), "-ldl"], check=True)
    _run(str(so), NO_CLUSTERS)
