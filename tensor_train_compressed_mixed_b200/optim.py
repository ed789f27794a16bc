"""AdamW: one optimiser step over many tensors in one launch, moments in 32 or 8 bits; the global gradient norm and
clipping by it, in place or within the step."""
from __future__ import annotations

import torch

from . import abi
from .dense import DenseEmbedding, on_device


def _trained(tables):
    """(parameters, gradients, guards) of TTEmbeddingBag and DenseEmbedding objects."""
    params, grads, guards = [], [], []
    for e in tables:
        if isinstance(e, DenseEmbedding):
            ps, gs, word = [e.table], [e.grad], abi.tt_emb_dense_status_word(e.handle)
        else:
            ps, gs, word = e.cores, e.grads, abi.tt_emb_status_word(e.handle)
        if ps is None or ps[0] is None or gs is None or gs[0] is None:
            raise ValueError("every table needs its cores (or table) and gradient buffers set")
        params += ps
        grads += gs
        guards += [word] * len(ps)
    return params, grads, guards


def _all_open(tables, of):
    for t in tables:
        if t.handle is None:
            raise ValueError(f"a table of this {of} has been closed")


class GradNorm:
    """The norm over the gradients of many tensors (root of the sum of all their squares), and clipping by it.

    grads: a list of contiguous CUDA tensors (float32, bfloat16 or float16), borrowed: they are read anew at every
    call.  guards: as AdamW's; a tensor whose guard is set counts as absent.  Calls of one object must be ordered (one
    stream, or events), replayed graphs that captured them included.  To clip before an AdamW step, give the bound to
    ``AdamW.step`` instead, which leaves the gradients as they are and reads them once less.
    """

    def __init__(self, grads, guards=None):
        grads = list(grads)
        if not grads:
            raise ValueError("grads must be a non-empty list")
        guards = [None] * len(grads) if guards is None else list(guards)
        if len(guards) != len(grads):
            raise ValueError("guards must have one entry for each tensor")
        self.device = grads[0].device if isinstance(grads[0], torch.Tensor) else None
        recs = []
        for i, (g, guard) in enumerate(zip(grads, guards)):
            if not isinstance(g, torch.Tensor) or not g.is_cuda or g.device != self.device:
                raise TypeError(f"grads[{i}] must be a CUDA tensor on the first one's device")
            if not g.is_contiguous():
                raise ValueError(f"grads[{i}] must be contiguous")
            recs.append(abi.NormTensor(grad=g.data_ptr(), guard=guard, size=g.numel(), grad_type=abi.dtype_code(g.dtype)))
        self.grads = grads
        self.tables = []
        with on_device(self.device):
            self.value = torch.zeros(1, dtype=torch.float32, device=self.device)
            torch.cuda.current_stream(self.device).synchronize()    # the first call may be given another stream
            self.handle = abi.tt_emb_norm_create(recs)

    @classmethod
    def for_tables(cls, tables):
        """Over the gradient buffers of TTEmbeddingBag and DenseEmbedding objects: those they have now.  A table whose
        backward reported a device error is left out until its next sync."""
        tables = list(tables)
        _, grads, guards = _trained(tables)
        self = cls(grads, guards=guards)
        self.tables = tables   # the guards are theirs
        return self

    def norm(self, stream=None) -> torch.Tensor:
        """The norm, as ``self.value``: a CUDA float32 tensor of one value that the next call overwrites."""
        _all_open(self.tables, "norm")
        with on_device(self.device):
            abi.tt_emb_norm_measure(self.handle, self.value, stream)
        return self.value

    def clip(self, max_norm: float, stream=None) -> torch.Tensor:
        """Multiplies every gradient by max_norm / norm where the norm is above max_norm (> 0), in place, and
        returns the norm before that, as ``norm`` does.  A norm that is not a number (an infinity or NaN in a
        gradient) leaves the gradients as they are.  Gradients that overlap each other cannot be clipped."""
        _all_open(self.tables, "norm")
        with on_device(self.device):
            abi.tt_emb_norm_clip(self.handle, max_norm, self.value, stream)
        return self.value

    def close(self):
        if getattr(self, "handle", None) is not None:
            abi.tt_emb_norm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class AdamW:
    """AdamW over contiguous CUDA tensors and their gradients (both borrowed: gradients are read
    from the buffers given here at every step).

    params, grads: lists of tensors of equal sizes, float32, bfloat16 or float16, no parameter on
    the memory of another or of a gradient; weight_decay: one number, or one for each tensor.
    state_bits 8 holds both moments as e4m3 codes with one float32 scale for each 256 values; the
    second one, held as its root, is rounded up or down at random from `seed`.  guards: for each
    tensor None or the address of a device status word, while which is not 0 the tensor is left as
    it is.

    The state is public and can be saved and put back: ``steps`` (int64 [1], on the device),
    and flat buffers ``m`` and ``v`` in which tensor i begins at ``offsets[i]``, with
    ``m_scale`` and ``v_scale`` in 8 bits (``v`` then holds roots).
    """

    def __init__(self, params, grads, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01,
                 state_bits: int = 32, seed: int = 0, guards=None):
        params, grads = list(params), list(grads)
        if not params or len(params) != len(grads):
            raise ValueError("params and grads must be non-empty lists of equal length")
        guards = [None] * len(params) if guards is None else list(guards)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * len(params)
        if len(guards) != len(params) or len(decay) != len(params):
            raise ValueError("guards and weight_decay must have one entry for each tensor")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        self.device = params[0].device if isinstance(params[0], torch.Tensor) else None
        for i, (p, g) in enumerate(zip(params, grads)):
            for t, name in ((p, f"params[{i}]"), (g, f"grads[{i}]")):
                if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != self.device:
                    raise TypeError(f"{name} must be a CUDA tensor on the first one's device")
                abi.dtype_code(t.dtype)
                if not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
            if p.numel() != g.numel():
                raise ValueError(f"params[{i}] has {p.numel()} values and its gradient {g.numel()}")
        self.params, self.grads = params, grads
        self.tables = []
        self.state_bits = state_bits
        B = abi.ADAMW_BLOCK
        self.offsets, total = [], 0
        for p in params:
            self.offsets.append(total)
            total += (p.numel() + B - 1) // B * B
        with on_device(self.device):
            self.steps = torch.zeros(1, dtype=torch.int64, device=self.device)
            self.norm = torch.zeros(1, dtype=torch.float32, device=self.device)
            kind = torch.float32 if state_bits == 32 else torch.uint8
            self.m = torch.zeros(total, dtype=kind, device=self.device)
            self.v = torch.zeros(total, dtype=kind, device=self.device)
            self.m_scale = self.v_scale = None
            if state_bits == 8:
                self.m, self.v = self.m.view(torch.float8_e4m3fn), self.v.view(torch.float8_e4m3fn)
                self.m_scale = torch.zeros(total // B, dtype=torch.float32, device=self.device)
                self.v_scale = torch.zeros(total // B, dtype=torch.float32, device=self.device)
            size = self.m.element_size()
            recs = []
            for p, g, at, guard, wd in zip(params, grads, self.offsets, guards, decay):
                r = abi.AdamWTensor(param=p.data_ptr(), grad=g.data_ptr(), exp_avg=self.m.data_ptr() + at * size,
                                    exp_avg_sq=self.v.data_ptr() + at * size, guard=guard, size=p.numel(),
                                    param_type=abi.dtype_code(p.dtype), grad_type=abi.dtype_code(g.dtype),
                                    weight_decay=float(wd))
                if state_bits == 8:
                    r.m_scale = self.m_scale.data_ptr() + at // B * 4
                    r.v_scale = self.v_scale.data_ptr() + at // B * 4
                recs.append(r)
            opt = abi.AdamWOptions(beta1=betas[0], beta2=betas[1], eps=eps, state_bits=state_bits,
                                   seed=seed & (2 ** 64 - 1))
            # the zeroed state is waited for: the first step may be given another stream
            torch.cuda.current_stream(self.device).synchronize()
            self.handle = abi.tt_emb_adamw_create(recs, opt, self.steps)

    @classmethod
    def for_tables(cls, tables, **options):
        """An optimiser of the cores and tables of TTEmbeddingBag and DenseEmbedding objects, whose
        gradient buffers it reads: those they have now, so make it after set_cores and set_table.
        A table whose backward reported a device error is left as it is until its next sync.

        Where several ranks train copies of the tables, the caller exchanges the gradients (a bag's
        ``grad_flat``, a dense table's ``grad``) before the step, and sees every rank's sync succeed first:
        a guard is this rank's own, and a rank whose backward failed would leave a table that the others
        update."""
        tables = list(tables)
        params, grads, guards = _trained(tables)
        self = cls(params, grads, guards=guards, **options)
        self.tables = tables   # the guards are theirs
        return self

    def step(self, lr, stream=None, max_norm=None):
        """One step of every tensor.  lr: a number, or a CUDA float32 tensor of one value, which a
        captured step reads anew at each replay.  Steps of one object must be ordered (one stream, or
        events), replayed graphs that captured them included.

        max_norm (> 0): the step's gradients are first multiplied by max_norm / norm where their global norm is above
        max_norm; the buffers keep what they hold.  Returns that norm then, as ``self.norm``: a CUDA float32 tensor of
        one value that the next such step overwrites.  A norm that is not a number (an infinity or NaN in a gradient)
        makes the step leave everything as it is, ``steps`` too."""
        _all_open(self.tables, "optimiser")
        if isinstance(lr, torch.Tensor) and lr.device != self.device:
            raise TypeError(f"lr must be a number or a tensor on {self.device}")
        with on_device(self.device):
            if max_norm is None:
                abi.tt_emb_adamw_step(self.handle, lr, stream)
                return None
            abi.tt_emb_adamw_step_clipped(self.handle, lr, max_norm, self.norm, stream)
        return self.norm

    def close(self):
        if getattr(self, "handle", None) is not None:
            abi.tt_emb_adamw_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
