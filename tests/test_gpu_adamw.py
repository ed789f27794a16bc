"""AdamW against the formulas in 64 bits (32-bit moments) and, code for code, against the 8-bit rule.

Tolerances of 32-bit moments count fp32 roundings of at most u = 2^-24 each: m is two constants,
two products and a sum (3u of the sum of its terms' magnitudes); v the same with g^2 (4u); the
update divides m by 1 - beta1^t and by the root, in which the correction of v, the root, eps and
expm1 enter: within 16u of lr |m terms| / denominator on top of m's own 3u; the weight takes 3u
for the decay factor, its product and the difference, and one rounding to its type.
"""
import numpy as np
import pytest
import torch

from tensor_train_compressed_mixed_b200 import AdamW, DenseEmbedding, abi, from_workload
from workloads import random_workload

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24
B1, B2, EPS = 0.9, 0.999, 1e-8


def _tensors(sizes, ptype, gtype, seed=0, shift=0):
    """Weights and gradients of the given sizes; shift moves each off its 16-byte place."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = lambda n, t, sd: (torch.randn(n + shift, generator=g, device="cuda") * sd).to(t)[shift:]  # noqa: E731
    return [make(n, ptype, 0.5) for n in sizes], [make(n, gtype, 0.1) for n in sizes]


def _fill(o, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for i, p in enumerate(o.params):
        cut = slice(o.offsets[i], o.offsets[i] + p.numel())
        o.m[cut] = torch.randn(p.numel(), generator=g, device="cuda") * 0.03
        o.v[cut] = torch.rand(p.numel(), generator=g, device="cuda") * 0.01


def _check32(p0, g0, m0, v0, p, m, v, t, lr, wd):
    p0, g0, m0, v0 = (x.double().cpu() for x in (p0, g0, m0, v0))
    m1, v1 = B1 * m0 + (1 - B1) * g0, B2 * v0 + (1 - B2) * g0 * g0
    terms = B1 * m0.abs() + (1 - B1) * g0.abs()
    den = (v1 / (1 - B2 ** t)).sqrt() + EPS
    want = p0 * (1 - lr * wd) - lr * m1 / (1 - B1 ** t) / den
    assert ((m.double().cpu() - m1).abs() <= 3 * U * terms + 1e-45).all()
    assert ((v.double().cpu() - v1).abs() <= 4 * U * v1 + 1e-45).all()
    half = torch.finfo(p.dtype).eps / 2 if p.dtype != F32 else 0.0
    tol = 3 * U * p0.abs() + 19 * U * lr * terms / (1 - B1 ** t) / den + U * want.abs()
    tol = tol + half * 1.001 * want.abs() + (2.0 ** -25 if p.dtype == F16 else 1e-40)
    assert ((p.double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("ptype,gtype", [(F32, F32), (BF16, BF16), (F16, F16), (F32, BF16), (BF16, F32), (F16, BF16), (F32, F16)])
@pytest.mark.parametrize("t0,shift", [(0, 0), (1000, 0), (10 ** 7, 0), (5, 1), (5, 3)])
def test_step_32(ptype, gtype, t0, shift):
    sizes = [1, 7, 255, 256, 257, 4099, 100003]
    ps, gs = _tensors(sizes, ptype, gtype, shift=shift)
    wd = [0.1 * (i % 2) for i in range(len(sizes))]
    o = AdamW(ps, gs, betas=(B1, B2), eps=EPS, weight_decay=wd)
    if t0:
        _fill(o)
    o.steps.fill_(t0)
    before = [[x.clone() for x in (p, g, o.m[a:a + p.numel()], o.v[a:a + p.numel()])] for p, g, a in zip(ps, gs, o.offsets)]
    o.step(0.01)
    assert int(o.steps) == t0 + 1
    lr = float(np.float32(0.01))
    for (p0, g0, m0, v0), p, a, w in zip(before, ps, o.offsets, wd):
        n = p.numel()
        _check32(p0, g0, m0, v0, p, o.m[a:a + n], o.v[a:a + n], t0 + 1, lr, w)
        end = a + -(-n // 256) * 256
        assert not o.m[a + n:end].any() and not o.v[a + n:end].any()     # behind a tensor nothing is written


def test_many_tensors_and_mixed_types_take_one_step():
    kinds = [(F32, F32), (BF16, BF16), (BF16, F32)]
    ps, gs = [], []
    for i in range(300):
        p, g = _tensors([i % 37 * 11], *kinds[i % 3], seed=i)
        ps, gs = ps + p, gs + g
    o = AdamW(ps, gs, weight_decay=0.0)
    before = [p.clone() for p in ps]
    zero = torch.zeros(1, device="cuda")
    o.step(0.01)
    assert int(o.steps) == 1
    for p0, p, g, a in zip(before, ps, gs, o.offsets):
        n = p.numel()
        if n:
            _check32(p0, g, zero.expand(n), zero.expand(n), p, o.m[a:a + n], o.v[a:a + n], 1, float(np.float32(0.01)), 0.0)


def test_only_empty_tensors_still_count_a_step():
    x = torch.empty(0, device="cuda")
    o = AdamW([x], [x])
    o.step(0.1)
    o.step(0.1)
    assert int(o.steps) == 2


# --------------------------------------------------------------------------- 8 bits
def _decode_table():
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()


def _mix(z):
    z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    return z ^ (z >> np.uint64(31))


def _rule8(p, g, mc, vc, ms, vs, first, t, lr, wd, seed):
    """The header's 8-bit rule in numpy float32, operation by operation; all arrays of whole blocks."""
    f = np.float32
    dec = _decode_table()
    with np.errstate(all="ignore"):
        m = dec[mc] * np.repeat(ms, 256)
        u = dec[vc] * np.repeat(vs, 256)
        v = u * u
        m = m * f(B1) + g * f(1 - B1)
        v = v * f(B2) + (g * g) * f(1 - B2)
        u = np.sqrt(v)
        m64, u64 = m.astype(np.float64), u.astype(np.float64)
        want = p.astype(np.float64) * (1 - lr * wd) - lr * m64 / (1 - B1 ** t) / (u64 / np.sqrt(1 - B2 ** t) + EPS)

        def top(x):
            a = np.abs(x).reshape(-1, 256)
            a = np.where(np.isfinite(a), a, 0).max(1).astype(f)
            return np.where(a < f(2.0 ** -100), f(0), a)

        am, au = top(m), top(u)
        im, iu = (np.where(a > 0, f(448) * (f(1) / np.where(a > 0, a, f(1))), f(0)).astype(f) for a in (am, au))
        x = np.where(np.isfinite(m), np.clip(m * np.repeat(im, 256), -448, 448), np.nan).astype(f)
        mcode = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        gamma = np.uint64(0x9E3779B97F4A7C15)
        start = _mix(np.array([t], np.uint64) * gamma + np.uint64(seed))
        q = np.uint64(first // 4) + np.arange(len(m) // 4, dtype=np.uint64) + np.uint64(1)
        word = _mix(start + q * gamma)
        part = np.stack([(word >> np.uint64(k)) & np.uint64(0xFFFF) for k in (0, 16, 32, 48)], 1).reshape(-1).astype(np.uint32)
        y = np.minimum(u * np.repeat(iu, 256), f(448)).astype(f) * f(2.0 ** -120)
        code = (y.view(np.uint32) + (part << np.uint32(4))) >> np.uint32(20)
        code = np.where(u > 0, np.maximum(code, 1), 0)
        code = np.where(np.isfinite(u), code, 0x7F).astype(np.uint8)
    return want, m, mcode, code, am * (f(1) / f(448)), au * (f(1) / f(448))


def _pad(x, n):
    return np.concatenate([x, np.zeros(n - len(x), x.dtype)])


def _check8(o, before, t, lr, wd, seed):
    for i, (p0, g, mc, vc, ms, vs) in enumerate(before):
        n = p0.numel()
        a, w = o.offsets[i], -(-n // 256) * 256
        b = slice(a // 256, a // 256 + w // 256)
        num = lambda x: _pad(x.float().cpu().numpy(), w)  # noqa: E731
        want, m, mcode, vcode, mscale, vscale = _rule8(num(p0), num(g), _pad(mc, w), _pad(vc, w), ms, vs, a, t, lr, wd, seed)
        got = lambda x: x.view(torch.uint8)[a:a + n].cpu().numpy()  # noqa: E731
        isnan = lambda c: (c & 0x7F) == 0x7F  # noqa: E731
        gm, gv = got(o.m), got(o.v)
        assert np.array_equal(isnan(gm), isnan(mcode[:n])) and np.array_equal(gm[~isnan(gm)], mcode[:n][~isnan(gm)])
        assert np.array_equal(gv, vcode[:n])
        assert np.array_equal(o.m_scale[b].cpu().numpy(), mscale) and np.array_equal(o.v_scale[b].cpu().numpy(), vscale)
        p = o.params[i].double().cpu().numpy()
        fine = np.isfinite(want[:n])
        half = 0.0 if o.params[i].dtype == F32 else torch.finfo(o.params[i].dtype).eps / 2
        upd = np.abs(want - num(p0).astype(np.float64) * (1 - lr * wd))[:n]
        tol = 4 * U * np.abs(num(p0)[:n]) + 17 * U * upd + (half * 1.001 + U) * np.abs(want[:n]) + (2.0 ** -25 if half == 2.0 ** -11 else 1e-40)
        assert np.all(np.abs(p - want[:n])[fine] <= tol[fine])
        assert np.array_equal(np.isfinite(p), fine)


def _snapshot(o):
    got = []
    for p, g, a in zip(o.params, o.grads, o.offsets):
        n = p.numel()
        b = slice(a // 256, a // 256 + -(-n // 256))
        code = lambda x: x.view(torch.uint8)[a:a + n].cpu().numpy()  # noqa: E731
        got.append((p.clone(), g.clone(), code(o.m), code(o.v), o.m_scale[b].cpu().numpy(), o.v_scale[b].cpu().numpy()))
    return got


@pytest.mark.parametrize("ptype,gtype,shift", [(F32, F32, 0), (BF16, BF16, 0), (F16, F16, 0), (BF16, F32, 1), (F32, BF16, 3)])
def test_steps_8(ptype, gtype, shift):
    sizes = [1, 9, 256, 300, 4100, 70001]
    ps, gs = _tensors(sizes, ptype, gtype, shift=shift)
    seed = 2 ** 63 + 12345
    o = AdamW(ps, gs, betas=(B1, B2), eps=EPS, weight_decay=0.1, state_bits=8, seed=seed)
    for t in range(1, 5):
        before = _snapshot(o)
        o.step(0.01)
        _check8(o, before, t, float(np.float32(0.01)), 0.1, seed)
        assert int(o.steps) == t
        for g in gs:
            g.mul_(-0.7)


def test_8_bit_edges():
    """Zero blocks, tiny and huge gradients, one value far above its block, and values that are not finite."""
    n = 256 * 8
    g = torch.zeros(n, device="cuda")
    g[256:512] = 1e-25
    g[512:768] = torch.linspace(1e-12, 1, 256, device="cuda")
    g[768] = 1e15
    g[769:1024] = 1e-3
    g[1024:1280] = 1.0
    g[1100], g[1101], g[1102] = float("nan"), float("inf"), -float("inf")
    g[1300] = 3e38                                   # its square is infinite
    g[1536:1792] = 1e-38
    p = torch.ones(n, device="cuda")
    o = AdamW([p], [g], betas=(B1, B2), eps=EPS, weight_decay=0.0, state_bits=8, seed=5)
    for t in (1, 2, 3):
        before = _snapshot(o)
        o.step(0.01)
        _check8(o, before, t, float(np.float32(0.01)), 0.0, 5)
    bad = ~torch.isfinite(p)
    assert set(bad.nonzero().flatten().tolist()) <= {1100, 1101, 1102, 1300}
    assert (p[:256] == 1).all()
    assert torch.isfinite(o.v_scale).all() and torch.isfinite(o.m_scale).all()


def test_rounding_of_roots_is_even_handed():
    """4096 blocks whose second moment sits between two codes: the mean code is at its place within 6 sigma."""
    n, k = 256 * 4096, 4096 * 255
    g = torch.full((n,), 0.55, device="cuda")
    g[::256] = 1.0                                   # the largest of each block
    p = torch.zeros(n, device="cuda")
    o = AdamW([p], [g], betas=(B1, B2), state_bits=8, seed=11)
    o.step(0.0)
    code = o.v.view(torch.uint8).view(-1, 256)[:, 1:].double()
    root = np.sqrt(np.float32(0.001) * np.float32(0.55) ** 2) / np.sqrt(np.float32(0.001)) * 448   # 246.4: between 240 and 256
    where = (root - 240) / 16
    low = int(torch.tensor(240.0).to(torch.float8_e4m3fn).view(torch.uint8))
    assert set(code.unique().tolist()) == {float(low), float(low + 1)}
    sigma = np.sqrt(where * (1 - where) / k)
    assert abs(float(code.mean()) - low - where) <= 6 * sigma + 2.0 ** -16


def test_small_decay_is_not_lost_in_8_bits():
    """With no gradient v falls by 0.1 % a step, far below a code: the mean over many values follows it."""
    n = 256 * 1024
    g = torch.rand(n, device="cuda") + 0.5
    p = torch.zeros(n, device="cuda")
    o = AdamW([p], [g], betas=(B1, B2), state_bits=8, seed=3)
    o.step(0.0)
    value = lambda: ((o.v.float().view(-1, 256) * o.v_scale[:, None]) ** 2).double().mean()  # noqa: E731
    first = float(value())
    g.zero_()
    for _ in range(200):
        o.step(0.0)
    # the rounding of roots adds at most a quarter of a step squared, 2^-8 of v, once for each code passed
    assert abs(float(value()) / first / 0.999 ** 200 - 1) < 0.03


# --------------------------------------------------------------------------- use
def test_lr_from_the_device_and_replay():
    p, g = torch.ones(5000, device="cuda"), torch.randn(5000, device="cuda")
    q = p.clone()
    a, b = AdamW([p], [g]), AdamW([q], [g])
    lr = torch.tensor([0.1], device="cuda")
    a.step(0.0)
    b.step(0.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(lr)
    assert int(a.steps) == 1                         # capturing runs nothing
    for x in (0.1, 0.02, 0.5):
        lr.fill_(x)
        graph.replay()
        b.step(x)
        assert torch.equal(p, q) and torch.equal(a.m, b.m) and torch.equal(a.v, b.v)
    assert int(a.steps) == 4


def test_lr_of_zero_moves_nothing():
    p = torch.randn(600, device="cuda")
    before, g = p.clone(), torch.randn(600, device="cuda")
    g[5], g[7] = 0.0, 1e30
    for bits in (32, 8):
        o = AdamW([p], [g], state_bits=bits)
        for lr in (0.0, 1e-38, torch.tensor([0.0], device="cuda"), torch.tensor([-1.0], device="cuda"), torch.tensor([float("nan")], device="cuda")):
            o.step(lr)
            # the infinite v of value 7 is NaN in 8 bits, and its weight with it from the next step on
            rest = [i for i in range(600) if bits == 32 or i != 7]
            assert torch.equal(p[rest], before[rest])
        assert int(o.steps) == 5


def test_tiny_eps_and_untouched_weights():
    """Weights that never had a gradient stay where they are, whatever eps."""
    p = torch.randn(600, device="cuda")
    before, g = p.clone(), torch.zeros(600, device="cuda")
    g[300:] = 1.0
    for bits in (32, 8):
        for eps in (1.2e-38, 1e-8, 1.0):
            o = AdamW([p], [g], eps=eps, weight_decay=0.0, state_bits=bits)
            for lr in (1e-3, 100.0):
                o.step(lr)
            assert torch.equal(p[:300], before[:300]) and torch.isfinite(p).all()


def test_state_can_be_saved_and_put_back():
    p, g = torch.randn(3000, device="cuda"), torch.randn(3000, device="cuda")
    for bits in (32, 8):
        o = AdamW([p], [g], state_bits=bits, seed=1)
        o.step(0.01)
        saved = [x.clone() for x in (p, o.m, o.v, o.steps) + ((o.m_scale, o.v_scale) if bits == 8 else ())]
        o.step(0.01)
        q = saved[0].clone()
        o2 = AdamW([q], [g], state_bits=bits, seed=1)
        for to, x in zip((o2.m, o2.v, o2.steps) + ((o2.m_scale, o2.v_scale) if bits == 8 else ()), saved[1:]):
            to.copy_(x)
        o2.step(0.01)
        assert torch.equal(p, q)


def test_offsets_beyond_32_bits():
    n = (1 << 32) + 1000
    p, g = torch.zeros(n, device="cuda", dtype=BF16), torch.zeros(n, device="cuda", dtype=BF16)
    for x in (g[:500], g[-700:]):
        x.fill_(1.0)
    o = AdamW([p], [g], state_bits=8, weight_decay=0.0)
    o.step(1.0)
    assert (p[:500] == -1).all() and (p[-700:] == -1).all() and not p[500:-700].any()


def test_refusals():
    p, g = torch.ones(8, device="cuda"), torch.ones(8, device="cuda")
    with pytest.raises(ValueError):
        AdamW([p], [g[:7]])
    with pytest.raises(ValueError):
        AdamW([torch.ones(16, device="cuda")[::2]], [g])
    with pytest.raises(TypeError):
        AdamW([p], [g.double()])
    with pytest.raises(TypeError):
        AdamW([p], [g.cpu()])
    with pytest.raises(abi.TTEmbError) as err:
        AdamW([p, p[2:]], [g, g[2:]])               # the same weights twice
    assert err.value.code == abi.TT_ERR_ARG
    table = DenseEmbedding(4, 4)
    table.set_table(torch.zeros(4, 4, device="cuda"))
    o = AdamW.for_tables([table])
    table.close()
    with pytest.raises(ValueError):
        o.step(0.1)
    with pytest.raises(ValueError):
        AdamW.for_tables([DenseEmbedding(4, 4)])    # no table set
    o = AdamW([p], [g])
    for lr in (-0.1, float("nan"), float("inf")):
        with pytest.raises(abi.TTEmbError) as err:
            o.step(lr)
        assert err.value.code == abi.TT_ERR_ARG
    for lr, kind in ((torch.ones(2, device="cuda"), ValueError), (torch.ones(1), TypeError), (torch.ones(1, device="cuda").double(), TypeError)):
        with pytest.raises(kind):
            o.step(lr)
    assert int(o.steps) == 0 and (p == 1).all()


def test_tables_train_together():
    """A compressed and a dense table, forward, backward and AdamW, three steps against 64 bits; then a bad
    token stops its own table's update only."""
    import oracle
    w = random_workload(71, (2, 2, 2), (1, 3, 3, 1), [(4, 5, 6), (3, 4, 5)], [110, 60], batch=9,
                        pooling={"kind": "uniform", "lo": 0, "hi": 5}, with_grad=True)
    bag, cores, idx, off = from_workload(w, with_grads=True)
    dense = DenseEmbedding(50, 24, scale=2.0, padding_idx=0)
    table = torch.randn(50, 24, device="cuda")
    dense.set_table(table)
    tok = torch.randint(50, (9, 7), device="cuda")
    up, up2 = torch.from_numpy(w.grad_out).cuda(), torch.randn(9, 7, 24, device="cuda")
    o = AdamW.for_tables([bag, dense], weight_decay=0.01)
    ref = [p.double().cpu() for p in o.params]
    ms, vs = [torch.zeros_like(p) for p in ref], [torch.zeros_like(p) for p in ref]
    lr = float(np.float32(0.01))
    for t in (1, 2, 3):
        bag.forward(idx, off, w.batch)
        dense.forward(tok)
        bag.backward(up)
        dense.backward(tok, up2)
        o.step(lr)
        w.cores = [[ref[k * 3 + j].float().numpy() for j in range(3)] for k in range(2)]
        grads = [torch.from_numpy(np.asarray(x)) for tab in oracle.workload_backward(w) for x in tab]
        keep = tok.cpu().flatten() != 0
        grads.append(torch.zeros(50, 24, dtype=torch.float64).index_add_(0, tok.cpu().flatten()[keep], up2.cpu().double().reshape(-1, 24)[keep]) * 2)
        for p, g, m, v, got in zip(ref, grads, ms, vs, o.params):
            m.mul_(B1).add_(g, alpha=1 - B1)
            v.mul_(B2).addcmul_(g, g, value=1 - B2)
            p.mul_(1 - lr * 0.01).sub_(lr * m / (1 - B1 ** t) / ((v / (1 - B2 ** t)).sqrt() + EPS))
            # gradients agree within 1e-4 normwise, so values of them below 1e-2 of the largest may move an
            # update by up to the whole step; the others by 1 % of it a step
            big = g.abs() > 1e-2 * g.abs().max()
            assert ((got.double().cpu() - p).abs() <= torch.where(big, 0.02 * lr * t, 2.0 * lr * t) + 1e-6).all()
    bag.sync()
    dense.sync()
    before = [p.clone() for p in o.params]
    bad = tok.clone()
    bad[3, 3] = 50
    dense.backward(bad, up2)
    o.step(lr)
    assert torch.equal(o.params[-1], before[-1]) and not torch.equal(o.params[0], before[0])
    with pytest.raises(abi.TTEmbError):
        dense.sync()
    dense.backward(tok, up2)
    o.step(lr)
    dense.sync()
    assert not torch.equal(o.params[-1], before[-1])
