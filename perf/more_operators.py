"""What is measured of the table's projection and of clipping by the global norm: cases, inputs, one pass, its work, and
its result in 64 bits.

Three families that a model's training and serving need around a dense table and its AdamW step:

* ``project`` and ``pgrad``: a dense table read as a matrix, out = act(x tableᵀ + bias) + residual (the output head
  that shares the token table, the projection of a narrow table to a model's width), and its gradients for x, the table
  and the bias (``DenseEmbedding.project`` and ``.project_backward``);
* ``clip``: the norm over all gradients, and the gradients scaled by it in place (``GradNorm.clip``);
* ``step``: an AdamW step on gradients clipped by their global norm (``AdamW.step`` with ``max_norm``).

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 256                      # values that share one scale of an 8-bit moment
BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.999, 1e-8, 1e-3, 0.01
M64 = (1 << 64) - 1
GOLDEN = 0x9E3779B97F4A7C15      # SplitMix64's increment and the two factors of its finaliser
MIX1, MIX2 = 0xBF58476D1CE4E5B9, 0x94D049BB133111EB


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _project(name, n, rows, dim, type_, out, act="none", cap=0.0, bias=False, residual=False, keep=False, extra=0):
    return {"name": name, "op": "project", "n": n, "rows": rows, "dim": dim, "type": type_, "out": out, "act": act, "cap": cap,
            "bias": bias, "residual": residual, "keep": keep, "extra": extra}


def _pgrad(name, n, rows, dim, type_, grad, act="none", cap=0.0, bias=False, accumulate=False, extra=0):
    return {"name": name, "op": "pgrad", "n": n, "rows": rows, "dim": dim, "type": type_, "grad": grad, "act": act, "cap": cap,
            "bias": bias, "accumulate": accumulate, "extra": extra}


def _clip(name, layout, count, least, most, grad, bound):
    return {"name": name, "op": "clip", "layout": layout, "count": count, "least": least, "most": most, "grad": grad, "bound": bound}


def _step(name, layout, count, least, most, param, grad, bits, steps, bound):
    return {"name": name, "op": "step", "layout": layout, "count": count, "least": least, "most": most, "param": param, "grad": grad,
            "bits": bits, "steps": steps, "bound": bound}


def listed():
    return [
        # logits of one generated token for each of eight sequences, by the token table, soft-capped
        _project("project_decode", 8, 32000, 4096, "bf16", "f32", act="softcap", cap=30.0),
        # logits of a training batch
        _project("project_train", 4096, 32000, 4096, "bf16", "bf16"),
        # a narrow factor of a table up to the model's width, what a training step keeps of it for its backward pass included
        _project("project_factor", 8192, 4096, 128, "f16", "f16", act="gelu", bias=True, residual=True, keep=True),
        # 32-bit operands of odd sizes, in wider buffers
        _project("project_odd", 1009, 4099, 515, "f32", "f32", act="silu", bias=True, residual=True, extra=3),
        # a small model's short batch
        _pgrad("pgrad_small", 200, 5000, 512, "bf16", "bf16", act="silu", bias=True),
        # a training batch's logits' gradients, into x and the token table
        _pgrad("pgrad_train", 4096, 32000, 4096, "bf16", "bf16"),
        # the narrow factor's
        _pgrad("pgrad_factor", 8192, 4096, 128, "f16", "f32", act="gelu", bias=True),
        # 32 bits, odd sizes, wider buffers, one of several micro-batches
        _pgrad("pgrad_odd", 301, 5003, 257, "f32", "f32", act="softcap", cap=30.0, bias=True, accumulate=True, extra=3),
        # norm weights and biases: many tiny tensors, latency
        _clip("clip_tiny", "spread", 40, 1, 4099, "f32", 0.5),
        # the gradients of the cores of 26 three-core tables of rank 64, before their SGD step
        _clip("clip_cores", "cores", 26, 46, 342, "f32", 0.5),
        # 16-bit weights of odd sizes with 8-bit moments, early in training, when gradients are clipped most
        _step("step_odd", "spread", 12, 1000, 2000003, "bf16", "bf16", 8, 3, 0.1),
        # the large matrices of a model and its token table, 8-bit moments
        _step("step_large", "even", 4, 96 << 20, 96 << 20, "bf16", "bf16", 8, 1000, 0.5),
    ]


def _span(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("project", "project", "pgrad", "pgrad", "clip", "step"))
    if op in ("clip", "step"):
        layout, count = rng.choice(("spread", "cores", "even")), _span(rng, 1, 26)
        least, most = (_span(rng, 4, 60), _span(rng, 60, 342)) if layout == "cores" else (_span(rng, 1, 5000), _span(rng, 5000, 8 << 20))
        grad, bound = rng.choice(("f32", "bf16", "f16")), rng.choice((0.01, 0.5, 0.9, 4.0))
        if op == "clip":
            c = _clip("", layout, count, least, most, grad, bound)
        else:
            c = _step("", layout, count, least, most, rng.choice(("f32", "bf16", "f16")), grad, rng.choice((32, 8)),
                      rng.choice((0, 1, 17, 1000, 123456)), bound)
    else:
        type_ = rng.choice(("f32", "bf16", "bf16", "f16"))
        while True:
            n, rows, dim = _span(rng, 1, 16384), _span(rng, 1, 131072), _span(rng, 1, 8192)
            if rng.random() < 0.5:
                rows, dim = max(8, rows // 8 * 8), max(8, dim // 8 * 8)
            if n * rows * dim <= 1 << (35 if type_ == "f32" else 37) and n * rows <= 1 << 27 and rows * dim <= 1 << 28:
                break
        act, extra = rng.choice(("none", "none", "relu", "gelu", "silu", "softcap")), rng.choice((0, 0, 8, 3))
        cap = rng.choice((5.0, 30.0)) if act == "softcap" else 0.0
        if op == "project":
            c = _project("", n, rows, dim, type_, rng.choice((type_, "f32")), act, cap, rng.random() < 0.5, rng.random() < 0.4,
                         rng.random() < 0.3, extra)
        else:
            c = _pgrad("", n, rows, dim, type_, rng.choice((type_, "f32")), act, cap, rng.random() < 0.5, rng.random() < 0.4, extra)
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


def _wide(g, n, dim, extra, dtype, sd=None):
    """An [n, dim] view of rows `extra` values further apart, as one part of a wider buffer has it."""
    x = torch.empty(n, dim + extra, device="cuda", dtype=dtype)
    return (x if sd is None else x.normal_(0, sd, generator=g))[:, :dim]


def _blocks_max(x):
    """Largest magnitude of each block."""
    a = x.abs().view(-1, BLOCK).amax(1)
    return torch.where(a < 2.0 ** -100, torch.zeros_like(a), a)


def _nearest8(x):
    a = _blocks_max(x)
    inv = torch.where(a > 0, 448.0 / a, torch.zeros_like(a))
    code = (x.view(-1, BLOCK) * inv[:, None]).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return code.view(-1), a * (1.0 / 448.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("clip", "step"):
        return _prepare_tensors(case, seed, g)
    n, rows, dim, extra, t = case["n"], case["rows"], case["dim"], case["extra"], TYPES[case["type"]]
    # hidden values behind a norm, and weights as they are initialised
    s = {"case": case, "x": _wide(g, n, dim, extra, t, 1.0),
         "table": torch.empty(rows, dim, device="cuda", dtype=t).normal_(0, 0.02, generator=g),
         "bias": torch.empty(rows, device="cuda").normal_(0, 0.1, generator=g) if case["bias"] else None,
         "act": None if case["act"] == "none" else case["act"], "cap": case["cap"] or None}
    if case["op"] == "project":
        out = TYPES[case["out"]]
        s["residual"] = _wide(g, n, rows, extra, out, 1.0) if case["residual"] else None
        s["out"] = _wide(g, n, rows, extra, out)
        s["pre"] = torch.empty(n, rows, device="cuda", dtype=out) if case["keep"] else None
    else:
        s["upstream"] = _wide(g, n, rows, extra, t, 1e-2)
        s["pre"] = _wide(g, n, rows, extra, t, 0.02 * math.sqrt(dim) + 0.1) if s["act"] else None
        s["grad"] = torch.empty(rows, dim, device="cuda", dtype=TYPES[case["grad"]]).normal_(0, 1e-2, generator=g)
        s["grad_x"] = torch.empty(n, dim, device="cuda", dtype=t)
        s["grad_bias"] = torch.empty(rows, device="cuda").normal_(0, 1e-2, generator=g) if case["bias"] else None
    if own:
        from tensor_train_compressed_mixed_b200 import DenseEmbedding
        e = DenseEmbedding(rows, dim, dtype=t)
        e.set_table(s["table"], grad=s.get("grad"), with_grad=case["op"] == "pgrad")
        s["emb"] = e
    return s


def _prepare_tensors(c, seed, g):
    sizes = _sizes(c)
    at, total = _places(sizes)
    real = torch.ones(total, device="cuda", dtype=torch.bool)
    for a, n in zip(at, sizes):
        real[a + n:a + -(-n // BLOCK) * BLOCK] = False

    def normal(dtype, sd):
        return torch.empty(total, device="cuda", dtype=dtype).normal_(0, sd, generator=g).mul_(real)

    s = {"case": c, "seed": seed % 1000003, "upstream": normal(TYPES[c["grad"]], 1e-3),
         "max_norm": c["bound"] * 1e-3 * math.sqrt(sum(sizes))}      # against the norm that such gradients have
    cut = lambda x: [x[a:a + n] for a, n in zip(at, sizes)]  # noqa: E731
    if c["op"] == "clip":
        if own:
            from tensor_train_compressed_mixed_b200 import GradNorm
            s["opt"] = GradNorm(cut(s["upstream"]))
        return s
    s["param"] = normal(TYPES[c["param"]], 0.02)
    s["steps"] = torch.full((1,), c["steps"], device="cuda", dtype=torch.int64)
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
        o = AdamW(cut(s["param"]), cut(s["upstream"]), betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, state_bits=c["bits"],
                  seed=s["seed"])
        for to, x in ((o.m, m), (o.v, v), (o.steps, s["steps"])):
            to.copy_(x)
        if c["bits"] == 8:
            o.m_scale.copy_(s["m_scale"])
            o.v_scale.copy_(s["v_scale"])
        s["opt"] = o
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    op = c["op"]
    if op == "project":
        return _run_project(s)
    if op == "pgrad":
        return _run_pgrad(s)
    # every pass is a step of its own, its bound a little lower, so that gradients clipped in place are clipped again
    bound = s["max_norm"]
    if op == "clip":
        s["max_norm"] *= 0.999
        if own:
            return [s["upstream"], s["opt"].clip(bound)]
        norm, by = _plain_norm(s["upstream"], bound)
        s["upstream"].copy_(s["upstream"].float() * by)
        return [s["upstream"], norm]
    if own:
        o = s["opt"]
        norm = o.step(LR, max_norm=bound)
        more = [o.m_scale, o.v_scale] if c["bits"] == 8 else []
        return [s["param"], o.m, o.v, o.steps, norm] + more
    return _plain_step(s, bound)


def _run_project(s):
    if own:
        out = s["emb"].project(s["x"], bias=s["bias"], activation=s["act"], cap=s["cap"], residual=s["residual"], out=s["out"],
                               pre=s["pre"])
        return [out] if s["pre"] is None else [out, s["pre"]]
    z = s["x"].float() @ s["table"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = z
    if s["act"] == "relu":
        y = torch.where(z > 0, z, torch.zeros_like(z))
    elif s["act"] == "gelu":
        y = 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    elif s["act"] == "silu":
        y = z / (1 + torch.exp(-z))
    elif s["act"] == "softcap":
        y = s["cap"] * torch.tanh(z / s["cap"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    s["out"].copy_(y)
    if s["pre"] is None:
        return [s["out"]]
    s["pre"].copy_(z)
    return [s["out"], s["pre"]]


def _run_pgrad(s):
    c = s["case"]
    if own:
        s["emb"].project_backward(s["x"], s["upstream"], pre=s["pre"], activation=s["act"], cap=s["cap"], accumulate=c["accumulate"],
                                  grad_x=s["grad_x"], grad_bias=s["grad_bias"])
        return [s["grad_x"], s["grad"]] + ([] if s["grad_bias"] is None else [s["grad_bias"]])
    d = s["upstream"].float()
    if s["act"]:
        z = s["pre"].float()
        if s["act"] == "relu":
            d = d * (z > 0)
        elif s["act"] == "gelu":
            d = d * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
        elif s["act"] == "silu":
            p = 1 / (1 + torch.exp(-z))
            d = d * (p * (1 + z * (1 - p)))
        else:
            t = torch.tanh(z / s["cap"])
            d = d * (1 - t * t)
    s["grad_x"].copy_(d @ s["table"].float())
    w = d.t() @ s["x"].float()
    s["grad"].copy_(s["grad"].float() + w if c["accumulate"] else w)
    if s["grad_bias"] is None:
        return [s["grad_x"], s["grad"]]
    b = d.double().sum(0)
    s["grad_bias"].copy_(s["grad_bias"] + b if c["accumulate"] else b)
    return [s["grad_x"], s["grad"], s["grad_bias"]]


def _plain_norm(g, bound):
    """The norm of all gradients, and the factor that takes it to the bound if it is above."""
    norm = torch.zeros((), device="cuda", dtype=torch.float64)
    for part in g.split(1 << 26):
        norm += part.double().square().sum()
    norm = norm.sqrt()
    return norm.float().view(1), torch.where(norm > bound, bound / norm, torch.ones_like(norm)).float()


def _plain_step(s, bound):
    c, p = s["case"], s["param"]
    norm, by = _plain_norm(s["upstream"], bound)
    s["steps"] += 1
    t = s["steps"].double()
    fix1, fix2 = (1 - BETA1 ** t).float(), (1 - BETA2 ** t).sqrt().float()
    g = s["upstream"].float() * by
    if c["bits"] == 8:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).square_().view(-1)
    else:
        m, v = s["m"], s["v"]
    m.mul_(BETA1).add_(g * (1 - BETA1))
    v.mul_(BETA2).add_(g * g * (1 - BETA2))
    root = v.sqrt()
    p.copy_(p.float() * (1 - LR * DECAY) - LR / fix1 * m / (root / fix2 + EPS))
    if c["bits"] == 32:
        return [p, m, v, s["steps"], norm]
    code, scale = _nearest8(m)
    s["m"].copy_(code)
    s["m_scale"].copy_(scale)
    code, scale = _random8(root, s["seed"], s["steps"])
    s["v"].copy_(code)
    s["v_scale"].copy_(scale)
    return [p, s["m"], s["v"], s["steps"], norm, s["m_scale"], s["v_scale"]]


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
def work(c):
    if c["op"] in ("clip", "step"):
        n = sum(_sizes(c))
        if c["op"] == "clip":
            return {"bytes": n * SIZE[c["grad"]] * (2 if c["bound"] < 1 else 1), "flops": 3.0 * n}
        state = 16 if c["bits"] == 32 else 4 + 16.0 / BLOCK
        return {"bytes": n * (2 * SIZE[c["param"]] + SIZE[c["grad"]] + state), "flops": 18.0 * n}
    n, rows, dim, size = c["n"], c["rows"], c["dim"], SIZE[c["type"]]
    if c["op"] == "project":
        moved = (n + rows) * dim * size + n * rows * SIZE[c["out"]] * (1 + c["residual"] + c["keep"]) + c["bias"] * rows * 4
        return {"bytes": moved, "flops": 2.0 * n * rows * dim}
    moved = (2 * n + rows) * dim * size + n * rows * size * (1 if c["act"] == "none" else 2)
    moved += rows * (dim * SIZE[c["grad"]] + c["bias"] * 4) * (1 + c["accumulate"])
    return {"bytes": moved, "flops": 4.0 * n * rows * dim}


# ---------------------------------------------------------------------------
# the same in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "project":
        return _exact_project(case, s)
    if case["op"] == "pgrad":
        return _exact_pgrad(case, s)
    g = s["upstream"]
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(x, dtype=torch.float64)) ** 2 for x in g.split(1 << 24)))
    by = min(1.0, s["max_norm"] / norm) if norm else 1.0
    told = torch.full((1,), norm, device="cuda", dtype=torch.float64)
    if case["op"] == "clip":
        return [g.double() * by, told]
    return _exact_step(case, s, by, told)


def _act64(case, z):
    if case["act"] == "relu":
        return z.clamp(min=0)
    if case["act"] == "gelu":
        return z * torch.special.ndtr(z)
    if case["act"] == "silu":
        return z * torch.sigmoid(z)
    return case["cap"] * torch.tanh(z / case["cap"]) if case["act"] == "softcap" else z


def _exact_project(case, s):
    """Some rows of x at a time."""
    w, out, pre = s["table"].double(), [], []
    bias = s["bias"].double() if case["bias"] else torch.zeros(case["rows"], device="cuda", dtype=torch.float64)
    for k in range(0, case["n"], 2048):
        z = torch.addmm(bias, s["x"][k:k + 2048].double(), w.t())
        pre.append(z if case["keep"] else None)
        y = _act64(case, z)
        out.append(y + s["residual"][k:k + 2048].double() if case["residual"] else y)
    return [torch.cat(out)] + ([torch.cat(pre)] if case["keep"] else [])


def _exact_pgrad(case, s):
    """The activation's slope by its own derivative in 64 bits, some rows at a time."""
    w = s["table"].double()
    dx, dw = [], torch.zeros(case["rows"], case["dim"], device="cuda", dtype=torch.float64)
    db = torch.zeros(case["rows"], device="cuda", dtype=torch.float64)
    for k in range(0, case["n"], 2048):
        d = s["upstream"][k:k + 2048].double()
        if case["act"] != "none":
            z = s["pre"][k:k + 2048].double().requires_grad_()
            d, = torch.autograd.grad(_act64(case, z), z, d)
        dx.append(d @ w)
        dw.addmm_(d.t(), s["x"][k:k + 2048].double())
        db += d.sum(0)
    if case["accumulate"]:
        dw += s["grad"].double()
        db += s["grad_bias"].double() if case["bias"] else 0
    return [torch.cat(dx), dw] + ([db] if case["bias"] else [])


def _exact_step(c, s, by, norm):
    """Moments and weights in 64 bits; 8-bit codes as the format's values: the nearest one for m, and for
    the root of v the one below or above, which the random bits choose."""
    t = c["steps"] + 1
    p, m, v = [], [], []
    m_scale, v_scale = [], []
    for lo in range(0, s["param"].numel(), 1 << 24):
        cut = slice(lo, lo + (1 << 24))
        g = s["upstream"][cut].double() * by
        m0, v0 = s["m"][cut].double(), s["v"][cut].double()
        if c["bits"] == 8:
            blocks = slice(lo // BLOCK, (lo + (1 << 24)) // BLOCK)
            m0 = m0 * s["m_scale"][blocks].double().repeat_interleave(BLOCK)
            v0 = (v0 * s["v_scale"][blocks].double().repeat_interleave(BLOCK)) ** 2
        m1, v1 = BETA1 * m0 + (1 - BETA1) * g, BETA2 * v0 + (1 - BETA2) * g * g
        hat = (m1 / (1 - BETA1 ** t)) / ((v1 / (1 - BETA2 ** t)).sqrt() + EPS)
        p.append(s["param"][cut].double() * (1 - LR * DECAY) - LR * hat)
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
    got = [torch.cat(x) for x in (p, m, v)] + [None, norm]
    return got + [torch.cat(m_scale), torch.cat(v_scale)] if c["bits"] == 8 else got


def _mixed_int(z):
    z = ((z ^ (z >> 30)) * MIX1) & M64
    z = ((z ^ (z >> 27)) * MIX2) & M64
    return z ^ (z >> 31)
