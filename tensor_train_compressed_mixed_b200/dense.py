"""DenseEmbedding: one dense table, its scaled lookup and its gradient.

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
