"""DenseEmbedding: one dense table, its scaled lookup, the table read as a matrix, and the gradients of both.

The tables that are not worth compressing (a model's token table, small categorical
ones) live beside the TT tables: same library, same streams, same errors.  As in
``embedding.py``, PyTorch supplies device memory and the current stream only.
"""
from __future__ import annotations

import contextlib

import torch

from . import abi

_HERE = contextlib.nullcontext()


def on_device(device: torch.device):
    """Makes `device` current for the library's calls where another one is."""
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def on_stream(stream):
    """Allocates on `stream` (a torch stream, its handle, or None for the current one), so that memory
    used there is not handed out again before work there has ended."""
    if stream is None:
        return _HERE
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class DenseEmbedding:
    """A table of num_rows rows of dim values (float32, bfloat16 or float16).

    ``forward`` returns scale * table[tokens]; ``backward`` the gradient of the table for an
    upstream gradient of those rows.  padding_idx: a row that receives no gradient.  Calls of one
    object must be ordered (one stream, or events), replayed graphs that captured them included.
    """

    def __init__(self, num_rows: int, dim: int, dtype: torch.dtype = torch.float32, scale: float = 1.0,
                 padding_idx: int | None = None, device="cuda"):
        if padding_idx is not None and not 0 <= padding_idx < num_rows:
            raise ValueError(f"padding_idx must be in [0, {num_rows}), got {padding_idx}")
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        with on_device(self.device):
            self.handle = abi.tt_emb_dense_create(num_rows, dim, dtype, scale,
                                                  -1 if padding_idx is None else padding_idx)
        self.num_rows, self.dim, self.dtype = int(num_rows), int(dim), dtype
        self.table = None
        self.grad = None
        self._ws = []           # the workspace in use is the last; captured calls keep using theirs
        self._ws_tokens = -1
        self._project_ws, self._project_bytes = None, 0     # the projection's workspace,
        self._project_ws_at = None                          # the stream that it was allocated on,
        self._project_kept = []                             # and those that captured calls use

    def _check(self, t, name: str, dtype=None):
        if not isinstance(t, torch.Tensor) or t.get_device() != self.device.index:   # -1 on the CPU
            raise TypeError(f"{name} must be a tensor on {self.device}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")

    def set_table(self, table: torch.Tensor, grad: torch.Tensor | None = None, with_grad: bool = True):
        """table: contiguous [num_rows, dim] (borrowed).  grad: a buffer for its gradient of the same
        shape, of any of the three types; allocated in the table's type if not given."""
        self._check(table, "table", self.dtype)
        if tuple(table.shape) != (self.num_rows, self.dim):
            raise ValueError(f"table has shape {tuple(table.shape)}")
        if grad is not None:
            self._check(grad, "grad")
            if tuple(grad.shape) != tuple(table.shape):
                raise ValueError(f"grad has shape {tuple(grad.shape)}")
        elif with_grad:
            grad = torch.empty_like(table)
        abi.tt_emb_dense_set_table(self.handle, table, grad)
        self.table, self.grad = table, grad

    def reserve(self, max_tokens: int, stream=None):
        """Allocates (or grows) the backward's workspace for up to this many tokens.

        Earlier, smaller ones live as long as the object, since a captured call goes on using the
        one that it was captured with; each is half as large again as the one before, at least."""
        if max_tokens <= self._ws_tokens:
            return
        if self._ws:
            max_tokens = min(max(max_tokens, self._ws_tokens * 3 // 2), 2 ** 31 - 2)
        nbytes = abi.tt_emb_dense_workspace_size(self.handle, max_tokens)
        with on_device(self.device), on_stream(stream):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        abi.tt_emb_dense_set_workspace(self.handle, ws, max_tokens)
        self._ws.append(ws)
        self._ws_tokens = max_tokens

    def forward(self, tokens: torch.Tensor, out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                stream=None) -> torch.Tensor:
        """scale * table[tokens], in out's type, or out_dtype, or the table's.

        out: rows of neighbouring values, all the same distance of at least dim values apart."""
        self._check(tokens, "tokens")
        with on_device(self.device):
            if out is None:
                with on_stream(stream):
                    out = torch.empty(*tokens.shape, self.dim, dtype=out_dtype or self.dtype, device=self.device)
            else:
                self._check(out, "out", out_dtype)
            abi.tt_emb_dense_forward(self.handle, tokens, out, self.dim, stream)
        return out

    def backward(self, tokens: torch.Tensor, grad_out: torch.Tensor, accumulate: bool = False,
                 stream=None) -> torch.Tensor:
        """The table's gradient for these tokens, written to (or added to) ``self.grad``."""
        self._check(tokens, "tokens")
        self._check(grad_out, "grad_out")
        with on_device(self.device):
            self.reserve(tokens.numel(), stream)
            abi.tt_emb_dense_backward(self.handle, tokens, grad_out, self.dim, accumulate, stream)
        return self.grad

    def _workspace(self, nbytes: int, stream, at: int):
        """A workspace of this size for a call of the projection on `stream`, whose handle is `at`.

        One that a captured call uses lives as long as the object; another until a larger one takes its place, which is half
        as large again, or by 64 MB if that is less."""
        last = self._project_bytes
        if nbytes > last:
            size = max(nbytes, last + min(last // 2, 64 << 20))
            with on_stream(stream):
                ws = torch.empty(size, dtype=torch.uint8, device=self.device)
            abi.tt_emb_dense_set_project_workspace(self.handle, ws)
            self._project_ws, self._project_bytes, self._project_ws_at = ws, size, at
        if stream is None:
            captured = torch._C._cuda_isCurrentStreamCapturing()
        else:
            with on_stream(stream):
                captured = torch._C._cuda_isCurrentStreamCapturing()
        if captured:
            if not self._project_kept or self._project_kept[-1] is not self._project_ws:
                self._project_kept.append(self._project_ws)
        elif at != self._project_ws_at:
            with on_stream(stream):
                self._project_ws.record_stream(torch.cuda.current_stream())

    def project(self, x: torch.Tensor, bias: torch.Tensor | None = None, activation: str | None = None,
                cap: float | None = None, residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                out_dtype: torch.dtype | None = None, pre: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """act(x tableᵀ + bias) + residual, in out's type, or out_dtype, or the table's: the output head that shares a
        token table, or a narrow table's rows at a model's width.  The table's scale does not enter.

        x: [..., dim], of the table's type.  bias: [num_rows].  activation: None, 'relu', 'gelu' (exact), 'silu', or
        'softcap', which is cap * tanh(z / cap).  residual, out: [..., num_rows]; residual may be out.  pre: a buffer of
        that shape that receives x tableᵀ + bias, which the backward of an activation wants.  All of these may be of any of the
        three types, and their rows may lie any one distance apart; no output may overlap another buffer."""
        for t, name, kind in ((x, "x", self.dtype), (bias, "bias", None), (residual, "residual", None), (pre, "pre", None),
                              (out, "out", out_dtype)):
            if t is not None or name == "x":
                self._check(t, name, kind)
        if x.dim() == 0 or x.size(-1) != self.dim:
            raise ValueError(f"x must hold rows of {self.dim} values, got {tuple(x.shape)}")
        with on_device(self.device):
            if out is None:
                with on_stream(stream):
                    out = torch.empty(*x.shape[:-1], self.num_rows, dtype=out_dtype or self.dtype, device=self.device)
            call = abi.project_call(x, self.num_rows, self.dim, out, bias, residual, pre, activation, cap)
            nbytes = abi.tt_emb_dense_project_workspace_size(self.handle, call)
            at = abi._stream_on(stream, self.device.index)
            if nbytes:
                self._workspace(nbytes, stream, at)
            abi.tt_emb_dense_project(self.handle, call, at)
        return out

    def project_backward(self, x: torch.Tensor | None, grad_out: torch.Tensor, pre: torch.Tensor | None = None,
                         activation: str | None = None, cap: float | None = None, accumulate: bool = False,
                         grad_x: torch.Tensor | bool = True, grad_bias: torch.Tensor | None = None,
                         table_grad: bool = True, stream=None):
        """The gradients of ``project`` for an upstream gradient grad_out [..., num_rows]: the table's, written to (or
        with accumulate added to) ``self.grad``, the bias's likewise to grad_bias if it is given, and x's, which is
        returned: in grad_x if that is a buffer, in a new tensor of the table's type, or not at all if it is False.

        pre: what ``project`` left there; not needed without an activation.  The residual's gradient is grad_out.
        grad_out, pre, grad_x, grad_bias and the table's gradient may each be of any of the three types.  A bfloat16 result beside a
        bfloat16 table may be formed from grad_out times the slope rounded to bfloat16; buffers of the other types get it in full.
        The table's padding row receives none.  table_grad=False leaves the table's out, and needs no x."""
        self._check(grad_out, "grad_out")
        if grad_out.dim() == 0 or grad_out.size(-1) != self.num_rows:
            raise ValueError(f"grad_out must hold rows of {self.num_rows} values, got {tuple(grad_out.shape)}")
        if table_grad:
            self._check(x, "x", self.dtype)
        for t, name in ((pre, "pre"), (grad_bias, "grad_bias")):
            if t is not None:
                self._check(t, name)
        with on_device(self.device):
            if grad_x is True:
                with on_stream(stream):
                    grad_x = torch.empty(*grad_out.shape[:-1], self.dim, dtype=self.dtype, device=self.device)
            elif grad_x is False:
                grad_x = None
            else:
                self._check(grad_x, "grad_x")
            call = abi.project_grad_call(x, self.num_rows, self.dim, grad_out, pre, activation, cap, grad_x, grad_bias, table_grad,
                                         accumulate)
            nbytes = abi.tt_emb_dense_project_backward_workspace_size(self.handle, call)
            at = abi._stream_on(stream, self.device.index)
            if nbytes:
                self._workspace(nbytes, stream, at)
            abi.tt_emb_dense_project_backward(self.handle, call, at)
        return grad_x

    def sync(self):
        with on_device(self.device):
            abi.tt_emb_dense_sync(self.handle)

    def close(self):
        if getattr(self, "handle", None) is not None:
            abi.tt_emb_dense_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
