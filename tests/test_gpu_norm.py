"""The global gradient norm, clipping by it and the clipped AdamW step against their formulas in 64 bits.

Tolerances count roundings: a group's squares are added in fp32, at most 32 of them, each off by half a step, the rest in fp64, and the
norm is rounded to fp32: (32 + 1) halves of 2^-23 of the sum, half of that for the root, and one more.  A clipped
gradient is off by that, by the factor's and the product's rounding, and by half a step of its type.
"""
import math

import pytest
import torch

from tensor_train_compressed_mixed_b200 import AdamW, DenseEmbedding, GradNorm, TTEmbError, abi

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24
NORM_TOL = 18 * U


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _least(dtype):
    return torch.finfo(dtype).smallest_normal * _half_step(dtype)


def _lists(kinds, sizes, shift=0, by=1.0, seed=1):
    """One tensor of each size, `shift` values behind a place that vectors can take."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        buf = torch.full((n + shift + 9,), 3.0, device="cuda", dtype=kinds[i % len(kinds)])
        buf[shift:shift + n] = (torch.randn(n, generator=g, device="cuda") * by).to(buf.dtype)
        out.append((buf, buf[shift:shift + n]))
    return [b for b, _ in out], [x for _, x in out]


def _norm64(grads):
    return math.sqrt(math.fsum(float(x.double().square().sum()) for x in grads))


SIZES = [[1], [0, 3], [1, 2, 3, 5, 7, 8, 15, 16, 17, 31, 33], [1000, 4099, 1], [8192, 8191, 16385], [300000, 17, 5000001], [100] * 300]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("kinds", [[F32], [BF16], [F16], [F32, F16, BF16]], ids=["f32", "bf16", "f16", "mixed"])
@pytest.mark.parametrize("shift", [0, 1, 5])
def test_norm_and_clip(sizes, kinds, shift):
    bufs, grads = _lists(kinds, sizes, shift, by=0.1)
    want = _norm64(grads)
    o = GradNorm(grads)
    got = o.norm()
    assert got.dtype == F32 and got.shape == (1,)
    assert abs(float(got) - want) <= NORM_TOL * want
    before = [x.clone() for x in grads]
    assert abs(float(o.clip(2 * want)) - want) <= NORM_TOL * want
    assert all(torch.equal(a, b) for a, b in zip(before, grads))          # below the bound: as they were
    o.clip(math.inf)
    assert all(torch.equal(a, b) for a, b in zip(before, grads))
    bound = 0.3 * want
    assert abs(float(o.clip(bound)) - want) <= NORM_TOL * want
    for was, now, buf in zip(before, grads, bufs):
        x = was.double() * 0.3
        assert ((now.double() - x).abs() <= (NORM_TOL + 4 * U + _half_step(now.dtype)) * x.abs() + _least(now.dtype)).all()
        assert (buf[:shift] == 3).all() and (buf[shift + now.numel():] == 3).all()
    again = [x.clone() for x in grads]
    for x, was in zip(grads, before):
        x.copy_(was)
    o.clip(bound)
    assert all(torch.equal(a, b) for a, b in zip(again, grads))           # the same bits


@pytest.mark.parametrize("kind,value", [(F32, 1e-30), (F32, 1e-42), (F32, 3e38), (F32, 1e25), (BF16, 1e-38), (BF16, 3e38), (F16, 6e-8), (F16, 65504.0),
                                        (F32, 2.0 ** -46), (F32, 2.0 ** 63)])
@pytest.mark.parametrize("n", [1, 1000, 70001])
def test_the_whole_range_of_the_types(kind, value, n):
    x = torch.full((n,), value, device="cuda").to(kind)
    x[::3] = 0
    small = torch.full((100,), 1e-20, device="cuda")        # beside values whose squares leave fp32
    o = GradNorm([x, small])
    want = _norm64([x, small])
    got = float(o.norm())
    assert got == math.inf if want >= 3.4028236e38 else abs(got - want) <= NORM_TOL * want + 2.0 ** -149
    before = x.clone()
    bound = float(torch.tensor(max(want / 2 if want < 1e38 else 1.0, 1e-44), dtype=torch.float32))
    o.clip(bound)
    w = before.double() * min(1.0, bound / want)
    # 1 / (1000 values of 3e38) is below 2^-126, where the factor's rounding to fp32 is half the least subnormal, 2^-150, and not
    # half a step of its value: 3e38 * 2^-150 = 2.1e-7 of a result of 0.04
    off = 2.0 ** -150 * before.double().abs()
    assert ((x.double() - w).abs() <= (NORM_TOL + 4 * U + _half_step(kind)) * w.abs() + off + 4 * _least(kind)).all()


def test_zeros_and_empty_lists():
    x = torch.zeros(5000, device="cuda")
    for grads in ([x], [x[:0]], [x[:0], x]):
        o = GradNorm(grads)
        o.value.fill_(7)
        assert float(o.norm()) == 0 and float(o.clip(1.0)) == 0
    assert (x == 0).all()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("kind", [F32, BF16, F16])
@pytest.mark.parametrize("at", [0, 777, -1])
def test_a_norm_that_is_not_a_number_changes_nothing(bad, kind, at):
    _, grads = _lists([kind], [1001, 20000])
    grads[1][at] = bad
    keep = [x.clone() for x in grads]
    o = GradNorm(grads)
    assert not math.isfinite(float(o.clip(1e-3)))
    params = [torch.ones(x.numel(), device="cuda") for x in grads]
    for bits in (32, 8):
        a = AdamW(params, grads, state_bits=bits)
        a.step(0.1, max_norm=1.0)
        assert not math.isfinite(float(a.norm)) and int(a.steps) == 0
        assert all((p == 1).all() for p in params) and not a.m.float().any() and not a.v.float().any()
    for x, y in zip(grads, keep):
        assert torch.equal(x.view(torch.int16 if kind != F32 else torch.int32), y.view(torch.int16 if kind != F32 else torch.int32))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", [F32, BF16, F16])
@pytest.mark.parametrize("sizes", [[1], [300, 4097, 20011], [64] * 200])
def test_clipped_step_is_the_step_of_clipped_gradients(bits, kind, sizes):
    """Against AdamW.step on gradients that hold factor * g in fp32, bit for bit; and without a bound that bites,
    against the step without one."""
    _, grads = _lists([kind], sizes, by=0.1, seed=5)
    want = _norm64(grads)
    for bound in (0.25 * want, 4 * want):
        g = torch.Generator(device="cuda").manual_seed(2)
        ps = [torch.randn(x.numel(), generator=g, device="cuda").to(kind) for x in grads]
        qs = [p.clone() for p in ps]
        a = AdamW(ps, grads, state_bits=bits, seed=9)
        keep = [x.clone() for x in grads]
        norm = None
        fs = []
        for _ in range(3):
            norm = a.step(1e-2, max_norm=bound)
            fs.append(norm.clone())
        assert norm is a.norm and abs(float(norm) - want) <= NORM_TOL * want
        assert all(torch.equal(x, y) for x, y in zip(keep, grads))
        # the factor: the nearest fp32 value to bound / norm; the norm in 64 bits is not told, so both neighbours are tried
        fit = False
        mid = torch.tensor(min(1.0, float(torch.tensor(bound, dtype=F32)) / want), dtype=F32)
        for by in (mid, torch.nextafter(mid, torch.tensor(0.0)), torch.nextafter(mid, torch.tensor(1.0))):
            rs = [q.clone() for q in qs]
            b = AdamW(rs, [(x.float() * by.cuda()) for x in keep], state_bits=bits, seed=9)
            for _ in range(3):
                b.step(1e-2)
            same = all(torch.equal(x, y) for x, y in zip(ps, rs)) and torch.equal(a.m.view(torch.uint8), b.m.view(torch.uint8)) and \
                torch.equal(a.v.view(torch.uint8), b.v.view(torch.uint8)) and int(b.steps) == int(a.steps) == 3
            fit = fit or same
        assert fit


def test_guards_leave_a_table_out():
    tables = []
    for k in range(2):
        e = DenseEmbedding(50, 8)
        e.set_table(torch.ones(50, 8, device="cuda"), grad=torch.full((50, 8), 1.0 + k, device="cuda"))
        tables.append(e)
    o, a = GradNorm.for_tables(tables), AdamW.for_tables(tables, weight_decay=0.0)
    assert abs(float(o.norm()) - math.sqrt(400 + 1600)) < 1e-4
    tables[0].forward(torch.tensor([50], device="cuda"))           # its later calls do nothing until the next sync
    tables[0].grad.fill_(math.nan)
    assert abs(float(o.clip(20.0)) - 40) < 1e-4
    assert (tables[1].grad - 1.0).abs().max() < 1e-6 and torch.isnan(tables[0].grad).all()
    assert abs(float(a.step(0.1, max_norm=1.0)) - 20) < 1e-4
    assert (tables[0].table == 1).all() and (tables[1].table != 1).all()
    with pytest.raises(TTEmbError):
        tables[0].sync()
    tables[0].close()
    for call in (o.norm, lambda: o.clip(1.0), lambda: a.step(0.1, max_norm=1.0)):
        with pytest.raises(ValueError):
            call()


def test_captured_and_on_other_streams():
    _, grads = _lists([F32, BF16], [5000, 70001, 3])
    params = [torch.ones(x.numel(), device="cuda") for x in grads]
    o, a = GradNorm(grads), AdamW(params, grads)
    start = [x.clone() for x in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o.clip(0.5, stream=side)
    side.synchronize()
    want = [x.clone() for x in grads]
    for x, y in zip(grads, start):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o.clip(0.5)
        a.step(0.01, max_norm=0.1)
    for _ in range(2):
        for x, y in zip(grads, start):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(grads, want))
        assert abs(float(a.norm) - 0.5) < 1e-3            # of bf16 gradients as clipping rounded them
    assert int(a.steps) == 2


def test_refusals():
    x = torch.zeros(8, device="cuda")
    with pytest.raises(TypeError):
        GradNorm([x, x.cpu()])
    with pytest.raises(ValueError):
        GradNorm([x[::2]])
    with pytest.raises(TypeError):
        GradNorm([x.double()])
    o = GradNorm([x, x[4:]])
    o.norm()
    with pytest.raises(TTEmbError) as e:
        o.clip(1.0)                                       # some values would be scaled twice
    assert e.value.code == abi.TT_ERR_ARG
    for bound in (0.0, -1.0, math.nan):
        with pytest.raises(TTEmbError):
            GradNorm([x]).clip(bound)
        with pytest.raises(TTEmbError):
            AdamW([x.clone()], [x]).step(0.1, max_norm=bound)


def test_more_than_32_bits_of_values():
    x = torch.zeros(2 ** 31 + 77, dtype=BF16, device="cuda")
    x[-3:] = 4.0
    x[5] = 3.0
    o = GradNorm([x])
    want = math.sqrt(3 * 16 + 9)
    assert abs(float(o.clip(want / 2)) - want) <= NORM_TOL * want
    assert x[-3:].tolist() == [2.0] * 3 and float(x[5]) == 1.5 and not x[6:-3].any()
