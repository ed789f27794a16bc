"""What is measured of the token-table and AdamW operators: cases, inputs, one pass, its work, and its result in 64 bits.

Two families that a trained embedding table needs beside its compressed neighbours:

* ``lookup`` and ``grad``: rows of a dense table, scaled, and the table's gradient
  (``DenseEmbedding.forward`` and ``.backward``);
* ``adamw``: one AdamW step over many tensors at once, moments in 32 bits, or in 8 bits with a
  scale for each block of 256 values (``AdamW.step``).

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 256                      # values that share one scale of an 8-bit moment
BETA1, BETA2, EPS, LR = 0.9, 0.999, 1e-8, 1e-3
M64 = (1 << 64) - 1
GOLDEN = 0x9E3779B97F4A7C15      # SplitMix64's increment and the two factors of its finaliser
MIX1, MIX2 = 0xBF58476D1CE4E5B9, 0x94D049BB133111EB


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _lookup(name, n, rows, dim, table, out, law="zipf", ids="i64", extra=0, scale=1.0):
    return {"name": name, "op": "lookup", "n": n, "rows": rows, "dim": dim, "table": table, "out": out, "law": law,
            "ids": ids, "extra": extra, "scale": scale}


def _grad(name, n, rows, dim, upstream, grad, law="zipf", ids="i64", extra=0, scale=1.0, pad=0.0, accumulate=False):
    return {"name": name, "op": "grad", "n": n, "rows": rows, "dim": dim, "upstream": upstream, "grad": grad, "law": law,
            "ids": ids, "extra": extra, "scale": scale, "pad": pad, "accumulate": accumulate}


def _adamw(name, layout, count, least, most, param, grad, bits, steps, decay=0.01):
    return {"name": name, "op": "adamw", "layout": layout, "count": count, "least": least, "most": most, "param": param,
            "grad": grad, "bits": bits, "steps": steps, "decay": decay}


def listed():
    return [
        # one generated token for each of eight sequences: latency
        _lookup("lookup_decode", 8, 32000, 4096, "bf16", "bf16", law="uniform", scale=64.0),
        # a prompt batch of natural text, rows scaled by the root of the width
        _lookup("lookup_prompt", 8192, 128000, 4096, "bf16", "bf16", scale=64.0),
        # an odd width, so that rows begin at 4-byte places, and 32-bit ids
        _lookup("lookup_odd", 30011, 100003, 129, "f32", "f32", law="uniform", ids="i32"),
        # a training batch from a 32-bit table into 16-bit activations, in a wider buffer
        _lookup("lookup_train", 131072, 256000, 2048, "f32", "bf16", extra=128),
        # a small model's step: the gradient of a short batch
        _grad("grad_small", 200, 5000, 512, "f32", "f32", law="uniform"),
        # a training batch of natural text over a large vocabulary, gradient overwritten
        _grad("grad_train", 32768, 128000, 4096, "bf16", "bf16", scale=64.0),
        # odd width, a padded batch (a third of the tokens), 16-bit upstream into 32 bits
        _grad("grad_padded", 10007, 50021, 515, "f16", "f32", pad=0.33, ids="i32"),
        # one of several micro-batches, added to what is there
        _grad("grad_accumulate", 65536, 256000, 2048, "bf16", "f32", accumulate=True),
        # norm weights and biases: many tiny tensors, latency
        _adamw("adamw32_tiny", "spread", 40, 1, 4099, "f32", "f32", 32, 0, decay=0.0),
        # the cores of 26 three-core tables of rank 64 (this repository's training step)
        _adamw("adamw32_cores", "cores", 26, 46, 342, "f32", "f32", 32, 1000),
        # 16-bit weights of odd sizes with 8-bit moments, early in training
        _adamw("adamw8_odd", "spread", 12, 1000, 2000003, "bf16", "bf16", 8, 3),
        # the large matrices of a model and its token table, 8-bit moments
        _adamw("adamw8_large", "even", 4, 96 << 20, 96 << 20, "bf16", "bf16", 8, 1000),
    ]


def _span(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("lookup", "lookup", "grad", "grad", "adamw", "adamw"))
    if op == "adamw":
        layout = rng.choice(("spread", "cores", "even"))
        bits = rng.choice((32, 8))
        count = _span(rng, 1, 26)
        least, most = (_span(rng, 4, 60), _span(rng, 60, 342)) if layout == "cores" else (_span(rng, 1, 5000), _span(rng, 5000, 8 << 20))
        c = _adamw("", layout, count, least, most, rng.choice(("f32", "bf16", "f16")), rng.choice(("f32", "bf16", "f16")), bits,
                   rng.choice((0, 1, 17, 1000, 123456)), rng.choice((0.0, 0.01, 0.1)))
    else:
        while True:
            n, rows, dim = _span(rng, 1, 131072), _span(rng, 1, 256000), _span(rng, 1, 8192)
            if rng.random() < 0.4:
                dim = max(8, dim // 8 * 8)
            if n * dim <= 1 << 27 and rows * dim <= 1 << 28:
                break
        law, ids = rng.choice(("zipf", "zipf", "uniform", "same")), rng.choice(("i64", "i32"))
        n = min(n, 8192) if law == "same" else n     # one row's sum of more terms is off in 32 bits, whatever adds it up
        extra, scale = rng.choice((0, 0, 8, 3)), rng.choice((1.0, 0.25, math.sqrt(dim)))
        if op == "lookup":
            c = _lookup("", n, rows, dim, rng.choice(("f32", "bf16", "f16")), rng.choice(("f32", "bf16")), law, ids, extra, scale)
        else:
            c = _grad("", n, rows, dim, rng.choice(("f32", "bf16")), rng.choice(("f32", "bf16")), law, ids, extra, scale,
                      rng.choice((0.0, 0.0, 0.5)), rng.random() < 0.4)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _sizes(c):
    """The tensors' sizes: even, spread over a range by their logarithm, or a three-core table's cores."""
    k, lo, hi = c["count"], c["least"], c["most"]
    at = [int(round(lo * (hi / lo) ** (i / max(1, k - 1)))) for i in range(k)]
    if c["layout"] == "cores":
        return [s for x in at for s in (x * 4 * 64, 64 * x * 4 * 64, 64 * x * 8)]
    return at


def _places(sizes):
    """First element of each tensor in one buffer, each a multiple of BLOCK, and the buffer's size."""
    at, total = [], 0
    for s in sizes:
        at.append(total)
        total += -(-s // BLOCK) * BLOCK
    return at, total


def _tokens(c, g):
    n, rows = c["n"], c["rows"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    if c["law"] == "uniform":
        t = (u * rows).long()
    elif c["law"] == "zipf":     # probability about 1 / rank, as words have, at ranks spread over the table
        rank = (torch.exp(u * math.log(rows + 1)) - 1).long().clamp_(0, rows - 1)
        step = next(p for p in (100003, 100019, 100043) if rows % p)
        t = (rank * step + 7) % rows
    else:
        t = torch.full((n,), int(torch.randint(rows, (1,), generator=g, device="cuda")), device="cuda")
    t = t.clamp_(0, rows - 1)
    if c.get("pad"):
        hit = torch.rand(n, generator=g, device="cuda") < c["pad"]
        t[hit] = _pad(c)
    return t.to(torch.int32 if c["ids"] == "i32" else torch.int64)


def _pad(c):
    return c["rows"] // 2 if c.get("pad") else None


def _wide(n, dim, extra, dtype):
    """An [n, dim] view of rows `extra` values apart, as one part of a wider buffer has it."""
    return torch.empty(n, dim + extra, device="cuda", dtype=dtype)[:, :dim]


def _blocks_max(x):
    """Largest finite magnitude of each block, spread to its values, and as one value each."""
    a = x.abs().view(-1, BLOCK)
    a = torch.where(torch.isfinite(a), a, torch.zeros_like(a)).amax(1)
    return torch.where(a < 2.0 ** -100, torch.zeros_like(a), a)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "adamw":
        return _prepare_adamw(case, seed, g)
    s = {"case": case, "tokens": _tokens(case, g), "scale": case["scale"], "pad": _pad(case)}
    rows, dim, n = case["rows"], case["dim"], case["n"]
    if case["op"] == "lookup":
        s["table"] = torch.empty(rows, dim, device="cuda", dtype=TYPES[case["table"]]).normal_(0, 0.02, generator=g)
        s["out"] = _wide(n, dim, case["extra"], TYPES[case["out"]])
    else:
        s["upstream"] = _wide(n, dim, case["extra"], TYPES[case["upstream"]])
        s["upstream"].copy_(torch.empty(n, dim, device="cuda", dtype=TYPES[case["upstream"]]).normal_(0, 1, generator=g))
        s["table"] = torch.empty(rows, dim, device="cuda", dtype=TYPES[case["grad"]])
        s["grad"] = torch.empty_like(s["table"]).normal_(0, 1, generator=g)
    if own:
        from tensor_train_compressed_mixed_b200 import DenseEmbedding
        e = DenseEmbedding(rows, dim, dtype=s["table"].dtype, scale=case["scale"], padding_idx=s["pad"])
        e.set_table(s["table"], grad=s.get("grad"), with_grad=case["op"] == "grad")
        if case["op"] == "grad":
            e.reserve(n)
        s["emb"] = e
    return s


def _prepare_adamw(c, seed, g):
    sizes = _sizes(c)
    at, total = _places(sizes)
    real = torch.ones(total, device="cuda", dtype=torch.bool)
    for a, n in zip(at, sizes):
        real[a + n:a + -(-n // BLOCK) * BLOCK] = False

    def normal(dtype, sd):
        return torch.empty(total, device="cuda", dtype=dtype).normal_(0, sd, generator=g).mul_(real)

    s = {"case": c, "seed": seed % 1000003, "param": normal(TYPES[c["param"]], 0.02), "upstream": normal(TYPES[c["grad"]], 1e-3),
         "steps": torch.full((1,), c["steps"], device="cuda", dtype=torch.int64)}
    if c["steps"]:
        m = normal(torch.float32, 3e-4)
        v = torch.rand(total, generator=g, device="cuda").mul_(real).add_(0.05).mul_(1e-6 * (1 - BETA2 ** c["steps"])).mul_(real)
    else:
        m, v = (torch.zeros(total, device="cuda") for _ in range(2))
    if c["bits"] == 8:
        m, s["m_scale"] = _nearest8(m)
        v, s["v_scale"] = _nearest8(v.sqrt_())
    s["m"], s["v"] = m, v
    if own:
        from tensor_train_compressed_mixed_b200 import AdamW
        cut = lambda x: [x[a:a + n] for a, n in zip(at, sizes)]  # noqa: E731
        o = AdamW(cut(s["param"]), cut(s["upstream"]), betas=(BETA1, BETA2), eps=EPS, weight_decay=c["decay"],
                  state_bits=c["bits"], seed=s["seed"])
        for to, x in ((o.m, m), (o.v, v), (o.steps, s["steps"])):
            to.copy_(x)
        if c["bits"] == 8:
            o.m_scale.copy_(s["m_scale"])
            o.v_scale.copy_(s["v_scale"])
        s["opt"] = o
    return s


def _nearest8(x):
    a = _blocks_max(x)
    inv = torch.where(a > 0, 448.0 / a, torch.zeros_like(a))
    code = (x.view(-1, BLOCK) * inv[:, None]).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return code.view(-1), a * (1.0 / 448.0)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        if op == "lookup":
            return s["emb"].forward(s["tokens"], out=s["out"])
        if op == "grad":
            return s["emb"].backward(s["tokens"], s["upstream"], accumulate=s["case"]["accumulate"])
        o = s["opt"]
        o.step(LR)
        more = [o.m_scale, o.v_scale] if s["case"]["bits"] == 8 else []
        return [s["param"], o.m, o.v, o.steps] + more
    if op == "lookup":
        s["out"].copy_(s["table"][s["tokens"]].float() * s["scale"])
        return s["out"]
    if op == "grad":
        g = s["upstream"].float() * s["scale"]
        if s["pad"] is not None:
            g = g * (s["tokens"] != s["pad"])[:, None]
        if s["case"]["accumulate"]:
            total = s["grad"].float()
        else:
            total = torch.zeros(s["grad"].shape, device="cuda", dtype=torch.float32)
        s["grad"].copy_(total.index_add_(0, s["tokens"], g))
        return s["grad"]
    return _plain_adamw(s)


def _plain_adamw(s):
    c, p = s["case"], s["param"]
    s["steps"] += 1
    t = s["steps"].double()
    fix1, fix2 = (1 - BETA1 ** t).float(), (1 - BETA2 ** t).sqrt().float()
    g = s["upstream"].float()
    if c["bits"] == 8:
        m = s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]
        v = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).square_()
        m, v = m.view(-1), v.view(-1)
    else:
        m, v = s["m"], s["v"]
    m.mul_(BETA1).add_(g * (1 - BETA1))
    v.mul_(BETA2).add_(g * g * (1 - BETA2))
    root = v.sqrt()
    p.copy_(p.float() * (1 - LR * c["decay"]) - LR / fix1 * m / (root / fix2 + EPS))
    if c["bits"] == 32:
        return [p, m, v, s["steps"]]
    code, scale = _nearest8(m)
    s["m"].copy_(code)
    s["m_scale"].copy_(scale)
    code, scale = _random8(root, s["seed"], s["steps"])
    s["v"].copy_(code)
    s["v_scale"].copy_(scale)
    return [p, s["m"], s["v"], s["steps"], s["m_scale"], s["v_scale"]]


def _signed(x):
    return x - (1 << 64) if x >> 63 else x


def _mix(z):
    """SplitMix64's finaliser on 64-bit words held as signed ones."""
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * _signed(MIX1)
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * _signed(MIX2)
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def _random8(u, seed, steps):
    """Roots in 8 bits, rounded up or down at random: the kept bits of u plus 16 random ones below them.

    Four values in a row take the four 16-bit parts of one output of SplitMix64, whose start is mixed
    from the seed and the step; a value above zero keeps the least code at least."""
    a = _blocks_max(u)
    inv = torch.where(a > 0, 448.0 / a, torch.zeros_like(a))
    x = (u.view(-1, BLOCK) * inv[:, None]).clamp_(max=448).view(-1)
    start = _mix(steps * _signed(GOLDEN) + seed)
    word = _mix(start + (torch.arange(u.numel() // 4, device="cuda") + 1) * _signed(GOLDEN))
    part = torch.stack([(word >> k) & 0xFFFF for k in (0, 16, 32, 48)], 1).view(-1).int()
    code = ((x * 2.0 ** -120).view(torch.int32) + part * 16) >> 20
    code = torch.where(u > 0, code.clamp_(min=1), code)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), a * (1.0 / 448.0)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _distinct(c, n):
    """Expected number of distinct rows among n tokens of the case's law."""
    rows = c["rows"]
    if c["law"] == "same":
        return min(1, n)
    if c["law"] == "uniform":
        return rows * -math.expm1(n * math.log1p(-1.0 / rows)) if rows > 1 else 1
    r = np.arange(1, rows + 1, dtype=np.float64)
    p = np.log1p(1 / r) / math.log(rows + 1)
    return float(-np.expm1(n * np.log1p(-np.minimum(p, 1 - 1e-12))).sum())


def work(c):
    if c["op"] == "adamw":
        n = sum(_sizes(c))
        state = 16 if c["bits"] == 32 else 4 + 16.0 / BLOCK
        return {"bytes": n * (2 * SIZE[c["param"]] + SIZE[c["grad"]] + state), "flops": 15.0 * n}
    n, dim = c["n"], c["dim"]
    ids = n * (4 if c["ids"] == "i32" else 8)
    if c["op"] == "lookup":
        return {"bytes": ids + _distinct(c, n) * dim * SIZE[c["table"]] + n * dim * SIZE[c["out"]], "flops": float(n * dim)}
    n *= 1 - c["pad"]
    rows = 2 * _distinct(c, n) if c["accumulate"] else c["rows"]
    return {"bytes": ids + n * dim * SIZE[c["upstream"]] + rows * dim * SIZE[c["grad"]], "flops": 2.0 * n * dim}


# ---------------------------------------------------------------------------
# the same in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lookup":
        return torch.nn.functional.embedding(s["tokens"], s["table"]).double().mul_(s["scale"])
    if case["op"] == "grad":
        return _exact_grad(case, s)
    return _exact_adamw(case, s)


def _exact_grad(c, s):
    """Row sums as differences of running sums over the tokens in sorted order, some columns at a time."""
    tok, order = torch.sort(s["tokens"].long(), stable=True)
    got = s["grad"].double() if c["accumulate"] else torch.zeros(c["rows"], c["dim"], device="cuda", dtype=torch.float64)
    ids, count = torch.unique_consecutive(tok, return_counts=True)
    last = count.cumsum(0)
    keep = torch.ones_like(ids, dtype=torch.bool) if s["pad"] is None else ids != s["pad"]
    for k in range(0, c["dim"], 256):
        run_ = s["upstream"][:, k:k + 256][order].double().cumsum(0)
        run_ = torch.cat([torch.zeros_like(run_[:1]), run_])
        part = (run_[last] - run_[last - count]) * s["scale"]
        got[ids[keep], k:k + 256] += part[keep]
    return got


def _exact_adamw(c, s):
    """Moments and weights in 64 bits; 8-bit codes as the format's values: the nearest one for m, and for
    the root of v the one below or above, which the random bits choose."""
    t = c["steps"] + 1
    p, m, v = [], [], []
    m_scale, v_scale = [], []
    for lo in range(0, s["param"].numel(), 1 << 24):
        cut = slice(lo, lo + (1 << 24))
        g = s["upstream"][cut].double()
        m0, v0 = s["m"][cut].double(), s["v"][cut].double()
        if c["bits"] == 8:
            blocks = slice(lo // BLOCK, (lo + (1 << 24)) // BLOCK)
            m0 = m0 * s["m_scale"][blocks].double().repeat_interleave(BLOCK)
            v0 = (v0 * s["v_scale"][blocks].double().repeat_interleave(BLOCK)) ** 2
        m1, v1 = BETA1 * m0 + (1 - BETA1) * g, BETA2 * v0 + (1 - BETA2) * g * g
        hat = (m1 / (1 - BETA1 ** t)) / ((v1 / (1 - BETA2 ** t)).sqrt() + EPS)
        p.append(s["param"][cut].double() * (1 - LR * c["decay"]) - LR * hat)
        if c["bits"] == 32:
            m.append(m1)
            v.append(v1)
            continue
        for x, to in ((m1, m), (v1.sqrt(), v)):
            top = x.abs().view(-1, BLOCK).amax(1).clamp_(min=2.0 ** -100)
            y = x / top.repeat_interleave(BLOCK) * 448
            least = torch.exp2(torch.floor(torch.log2(y.abs().clamp_(min=2.0 ** -6))) - 3)   # step of the format at y
            if to is m:
                to.append(torch.round(y / least) * least)
            else:
                z = torch.arange(lo // 4, (lo + x.numel()) // 4, device="cuda")
                start = _mixed_int((t * GOLDEN + s["seed"]) & M64)
                z = _mix(torch.full_like(z, _signed(start)) + (z + 1) * _signed(GOLDEN))
                part = torch.stack([(z >> k) % 65536 for k in (0, 16, 32, 48)], 1).view(-1).double() / 65536
                low = torch.floor(y / least)
                up = (y / least - low + part >= 1).double()
                to.append(torch.where(x > 0, ((low + up) * least).clamp_(min=2.0 ** -9), torch.zeros_like(x)))
            (m_scale if to is m else v_scale).append(torch.where(top > 2.0 ** -100, top, torch.zeros_like(top)) / 448)
    got = [torch.cat(x) for x in (p, m, v)] + [None]
    return got + [torch.cat(m_scale), torch.cat(v_scale)] if c["bits"] == 8 else got


def _mixed_int(z):
    z = ((z ^ (z >> 30)) * MIX1) & M64
    z = ((z ^ (z >> 27)) * MIX2) & M64
    return z ^ (z >> 31)
