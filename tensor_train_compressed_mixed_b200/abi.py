"""ctypes binding of libttemb (include/tt_emb.h): argument marshalling only.

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: tensors are checked for device, dtype and layout,
their pointers and the current CUDA stream are passed through, and a non-OK
status becomes a ``TTEmbError``.  There is no CPU path: without the built
library (``python -m tensor_train_compressed_mixed_b200.build``) importing
the functions raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

PKG = os.path.dirname(os.path.abspath(__file__))
# TTEMB_LIB names another build of the same library (e.g. a variant compiled for a comparison)
LIB_PATH = os.environ.get("TTEMB_LIB") or os.path.join(PKG, "libttemb.so")

TT_OK, TT_ERR_ARG, TT_ERR_SHAPE, TT_ERR_INDEX_RANGE, TT_ERR_OFFSETS = 0, 1, 2, 3, 4
TT_ERR_WORKSPACE, TT_ERR_STATE, TT_ERR_CUDA, TT_ERR_TIMEOUT, TT_ERR_UNSUPPORTED = 5, 6, 7, 8, 9
TT_SCHED_STATIC, TT_SCHED_STEAL, TT_SCHED_STEAL_L2 = 0, 1, 2
TT_GROUP_PREFIX, TT_GROUP_UNIQUE_ONLY = 0, 1
TT_PREC_FP32, TT_PREC_BF16_TC, TT_PREC_FP32_SPLIT_TC = 0, 1, 2
TT_INJECT_NONE, TT_INJECT_POOL_WAIT, TT_INJECT_MMA_WAIT_FWD, TT_INJECT_MMA_WAIT_BWD = 0, 1, 2, 3
TT_F32, TT_BF16, TT_F16 = 0, 1, 2
MAX_TABLES, MAX_CORES = 64, 4
ADAMW_BLOCK = 256      # values that share one scale of an 8-bit moment


class TTEmbError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {error_string(code)} (status {code})")


class Options(ctypes.Structure):
    _fields_ = [("sched", ctypes.c_int32), ("grouping", ctypes.c_int32),
                ("chunk", ctypes.c_int32), ("grid", ctypes.c_int32),
                ("force_generic", ctypes.c_int32), ("precision", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 10)]


class SegView(ctypes.Structure):
    _fields_ = [("num_lookups", ctypes.c_int64), ("num_unique", ctypes.c_int64),
                ("num_groups", ctypes.c_int64), ("key_bits", ctypes.c_int32),
                ("key_bytes", ctypes.c_int32), ("sorted_keys", ctypes.c_void_p),
                ("perm", ctypes.c_void_p), ("uniq_keys", ctypes.c_void_p),
                ("uniq_start", ctypes.c_void_p), ("grp_start", ctypes.c_void_p),
                ("bag_sorted", ctypes.c_void_p)]


class AdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("guard", ctypes.c_void_p), ("size", ctypes.c_int64), ("param_type", ctypes.c_int32),
                ("grad_type", ctypes.c_int32), ("weight_decay", ctypes.c_double)]


class AdamWOptions(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("state_bits", ctypes.c_int32), ("reserved", ctypes.c_int32), ("seed", ctypes.c_uint64)]


_LIB = None

_SIGS = {
    "tt_emb_abi_version": ([], ctypes.c_int),
    "tt_emb_default_options": ([ctypes.POINTER(Options)], None),
    "tt_emb_error_string": ([ctypes.c_int], ctypes.c_char_p),
    "tt_emb_create": ([ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                       ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Options),
                       ctypes.POINTER(ctypes.c_void_p)], ctypes.c_int),
    "tt_emb_set_cores": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "tt_emb_workspace_size": ([ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                               ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
    "tt_emb_set_workspace": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64,
                              ctypes.c_int64], ctypes.c_int),
    "tt_emb_forward": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                        ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "tt_emb_backward": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "tt_emb_sgd_update": ([ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p], ctypes.c_int),
    "tt_emb_backward_sgd": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p], ctypes.c_int),
    "tt_emb_get_segmentation": ([ctypes.c_void_p, ctypes.POINTER(SegView)], ctypes.c_int),
    "tt_emb_copy_segmentation": ([ctypes.c_void_p] + [ctypes.c_void_p] * 6, ctypes.c_int),
    "tt_emb_sync": ([ctypes.c_void_p], ctypes.c_int),
    "tt_emb_enable_timing": ([ctypes.c_void_p, ctypes.c_int], ctypes.c_int),
    "tt_emb_phase_times": ([ctypes.c_void_p, ctypes.POINTER(ctypes.c_double),
                            ctypes.POINTER(ctypes.c_int64)], ctypes.c_int),
    "tt_emb_forward_noalloc": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "tt_emb_last_error": ([ctypes.c_void_p], ctypes.c_int),
    "tt_emb_set_probe": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32], ctypes.c_int),
    "tt_emb_debug_inject": ([ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32], ctypes.c_int),
    "tt_emb_destroy": ([ctypes.c_void_p], None),
    "tt_emb_dense_create": ([ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_float, ctypes.c_int64,
                             ctypes.POINTER(ctypes.c_void_p)], ctypes.c_int),
    "tt_emb_dense_set_table": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32], ctypes.c_int),
    "tt_emb_dense_workspace_size": ([ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)],
                                    ctypes.c_int),
    "tt_emb_dense_set_workspace": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64],
                                   ctypes.c_int),
    "tt_emb_dense_forward": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p,
                              ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p], ctypes.c_int),
    "tt_emb_dense_backward": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p,
                               ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p], ctypes.c_int),
    "tt_emb_dense_sync": ([ctypes.c_void_p], ctypes.c_int),
    "tt_emb_dense_last_error": ([ctypes.c_void_p], ctypes.c_int),
    "tt_emb_dense_destroy": ([ctypes.c_void_p], None),
    "tt_emb_status_word": ([ctypes.c_void_p], ctypes.c_void_p),
    "tt_emb_dense_status_word": ([ctypes.c_void_p], ctypes.c_void_p),
    "tt_emb_adamw_create": ([ctypes.c_int32, ctypes.POINTER(AdamWTensor), ctypes.POINTER(AdamWOptions),
                             ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)], ctypes.c_int),
    "tt_emb_adamw_step": ([ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "tt_emb_adamw_destroy": ([ctypes.c_void_p], None),
}

NOALLOC_MAX_LOOKUPS = 262144

PHASES = ("fwd_keys", "fwd_sort", "fwd_segment", "fwd_fused", "bwd_fused", "bwd_reduce", "sgd",
          "bwd_rowsum")


def lib() -> ctypes.CDLL:
    """The loaded libttemb.so; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m tensor_train_compressed_mixed_b200.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(h, name)
            fn.argtypes = args
            fn.restype = res
        _LIB = h
    return _LIB


def error_string(code: int) -> str:
    return lib().tt_emb_error_string(int(code)).decode()


def _check(rc: int, where: str):
    if rc != TT_OK:
        raise TTEmbError(rc, where)


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _stream_on(stream, device: int) -> int:
    """The given stream, or the current one of device number `device`."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dev_ptr(t, dtype, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def tt_emb_abi_version() -> int:
    return lib().tt_emb_abi_version()


def tt_emb_default_options() -> Options:
    o = Options()
    lib().tt_emb_default_options(ctypes.byref(o))
    return o


def tt_emb_create(n_factors, n_rows, d_factors, ranks, options: Options | None = None):
    """n_factors: [T][k] ints; n_rows: [T]; d_factors: [k]; ranks: [k+1]. Returns a handle."""
    n = np.ascontiguousarray(np.asarray(n_factors, dtype=np.int64))
    if n.ndim != 2:
        raise ValueError("n_factors must be [T][k]")
    rows = np.ascontiguousarray(np.asarray(n_rows, dtype=np.int64).reshape(-1))
    d = np.ascontiguousarray(np.asarray(d_factors, dtype=np.int32).reshape(-1))
    r = np.ascontiguousarray(np.asarray(ranks, dtype=np.int32).reshape(-1))
    T, k = n.shape
    if rows.size != T or d.size != k or r.size != k + 1:
        raise ValueError("inconsistent table shapes")
    h = ctypes.c_void_p()
    opt = ctypes.byref(options) if options is not None else None
    _check(lib().tt_emb_create(T, k, n.ctypes.data, rows.ctypes.data, d.ctypes.data, r.ctypes.data,
                               opt, ctypes.byref(h)), "tt_emb_create")
    return h


def tt_emb_set_cores(h, cores, core_grads=None):
    """cores / core_grads: flat lists of T*k float32 CUDA tensors, table-major."""
    ptrs = (ctypes.c_void_p * len(cores))(*[_dev_ptr(c, torch.float32, "core").value for c in cores])
    gptrs = None
    if core_grads is not None:
        gptrs = (ctypes.c_void_p * len(core_grads))(
            *[_dev_ptr(g, torch.float32, "core_grad").value for g in core_grads])
    _check(lib().tt_emb_set_cores(h, ptrs, gptrs), "tt_emb_set_cores")


def tt_emb_workspace_size(h, max_lookups: int, batch: int) -> int:
    out = ctypes.c_size_t()
    _check(lib().tt_emb_workspace_size(h, int(max_lookups), int(batch), ctypes.byref(out)),
           "tt_emb_workspace_size")
    return int(out.value)


def tt_emb_set_workspace(h, workspace, max_lookups: int, batch: int):
    ptr = _dev_ptr(workspace, torch.uint8, "workspace")
    _check(lib().tt_emb_set_workspace(h, ptr, workspace.numel(), int(max_lookups), int(batch)),
           "tt_emb_set_workspace")


def tt_emb_forward(h, indices, offsets, batch: int, out, stream=None):
    _check(lib().tt_emb_forward(h, _dev_ptr(indices, torch.int64, "indices"),
                                _dev_ptr(offsets, torch.int64, "offsets"), indices.numel(),
                                int(batch), _dev_ptr(out, torch.float32, "out"), _stream(stream)),
           "tt_emb_forward")


def tt_emb_backward(h, grad_out, stream=None):
    _check(lib().tt_emb_backward(h, _dev_ptr(grad_out, torch.float32, "grad_out"), _stream(stream)),
           "tt_emb_backward")


def tt_emb_sgd_update(h, lr: float, stream=None):
    _check(lib().tt_emb_sgd_update(h, float(lr), _stream(stream)), "tt_emb_sgd_update")


def tt_emb_backward_sgd(h, grad_out, lr: float, stream=None):
    _check(lib().tt_emb_backward_sgd(h, _dev_ptr(grad_out, torch.float32, "grad_out"), float(lr),
                                     _stream(stream)), "tt_emb_backward_sgd")


def tt_emb_sync(h):
    _check(lib().tt_emb_sync(h), "tt_emb_sync")


def tt_emb_get_segmentation(h) -> SegView:
    v = SegView()
    _check(lib().tt_emb_get_segmentation(h, ctypes.byref(v)), "tt_emb_get_segmentation")
    return v


def tt_emb_copy_segmentation(h) -> dict:
    """The last forward's segmentation, copied to host numpy arrays."""
    v = tt_emb_get_segmentation(h)
    L, U, G = v.num_lookups, v.num_unique, v.num_groups
    kt = np.uint64 if v.key_bytes == 8 else np.uint32
    out = {
        "sorted_keys": np.zeros(L, kt), "perm": np.zeros(L, np.int32),
        "uniq_keys": np.zeros(U, kt), "uniq_start": np.zeros(U + 1, np.int32),
        "grp_start": np.zeros(G + 1, np.int32), "bag_sorted": np.zeros(L, np.int32),
    }
    _check(lib().tt_emb_copy_segmentation(
        h, out["sorted_keys"].ctypes.data, out["perm"].ctypes.data, out["uniq_keys"].ctypes.data,
        out["uniq_start"].ctypes.data, out["grp_start"].ctypes.data, out["bag_sorted"].ctypes.data),
        "tt_emb_copy_segmentation")
    if L == 0:
        out["uniq_start"][:] = 0
        out["grp_start"][:] = 0
    out.update(num_lookups=L, num_unique=U, num_groups=G, key_bits=v.key_bits)
    return out


def tt_emb_forward_noalloc(h, indices, offsets, batch: int, out, stream=None):
    """Forward pass using the library's fixed device scratch instead of a workspace."""
    _check(lib().tt_emb_forward_noalloc(h, _dev_ptr(indices, torch.int64, "indices"),
                                        _dev_ptr(offsets, torch.int64, "offsets"), indices.numel(),
                                        int(batch), _dev_ptr(out, torch.float32, "out"),
                                        _stream(stream)),
           "tt_emb_forward_noalloc")


def tt_emb_enable_timing(h, enable: bool = True):
    _check(lib().tt_emb_enable_timing(h, 1 if enable else 0), "tt_emb_enable_timing")


def tt_emb_phase_times(h):
    """(per-phase milliseconds as a dict, kernels launched) since timing was enabled."""
    ms = (ctypes.c_double * len(PHASES))()
    n = ctypes.c_int64()
    _check(lib().tt_emb_phase_times(h, ms, ctypes.byref(n)), "tt_emb_phase_times")
    return dict(zip(PHASES, list(ms))), int(n.value)


def tt_emb_last_error(h) -> int:
    """The most recent failure recorded on the handle (a status code), then cleared."""
    return int(lib().tt_emb_last_error(h))


def tt_emb_set_probe(h, records, max_blocks: int):
    """Balance probe: records is a CUDA int64 tensor of 2 * max_blocks * 4 entries, or None."""
    ptr = ctypes.c_void_p(0) if records is None else _dev_ptr(records, torch.int64, "records")
    _check(lib().tt_emb_set_probe(h, ptr, int(max_blocks) if records is not None else 0), "tt_emb_set_probe")


def tt_emb_debug_inject(h, what: int, spin_limit: int = 0):
    """Test hook: arms one injected failure of a bounded device wait (TT_INJECT_*)."""
    _check(lib().tt_emb_debug_inject(h, int(what), int(spin_limit)), "tt_emb_debug_inject")


def tt_emb_destroy(h):
    if h is not None and h.value:
        lib().tt_emb_destroy(h)


# ---------------------------------------------------------------------------
# Dense tables
# ---------------------------------------------------------------------------
_CODES = {torch.float32: TT_F32, torch.bfloat16: TT_BF16, torch.float16: TT_F16}


def dtype_code(dtype) -> int:
    """TT_F32, TT_BF16 or TT_F16 of a torch dtype."""
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    return code


def _tokens(t):
    """(pointer, bytes of a token, tokens) of an integer CUDA tensor of any shape."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("tokens must be a CUDA tensor")
    nbytes = 8 if t.dtype is torch.int64 else 4 if t.dtype is torch.int32 else 0
    if not nbytes:
        raise TypeError(f"tokens must be int32 or int64, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return t.data_ptr(), nbytes, t.numel()


def _rows(t, n: int, dim: int, name: str):
    """(pointer, type, row stride) of n rows of dim values, each of neighbouring values and all the same
    distance apart (0 for an expanded tensor)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    code = dtype_code(t.dtype)
    if t.numel() != n * dim or t.dim() == 0 or t.size(-1) != dim:
        raise ValueError(f"{name} must hold {n} rows of {dim} values, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), code, dim
    try:
        t = t.view(n, dim)
    except RuntimeError:
        raise ValueError(f"{name}'s rows must be the same distance apart") from None
    if dim > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return t.data_ptr(), code, t.stride(0)


def tt_emb_dense_create(num_rows: int, dim: int, dtype, scale: float = 1.0, padding_row: int = -1):
    h = ctypes.c_void_p()
    _check(lib().tt_emb_dense_create(int(num_rows), int(dim), dtype_code(dtype), float(scale), int(padding_row),
                                     ctypes.byref(h)), "tt_emb_dense_create")
    return h


def tt_emb_dense_set_table(h, table, grad=None):
    for t, name in ((table, "table"), (grad, "grad")):
        if t is not None and not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()):
            raise TypeError(f"{name} must be a contiguous CUDA tensor")
    _check(lib().tt_emb_dense_set_table(h, table.data_ptr(), None if grad is None else grad.data_ptr(),
                                        dtype_code(table.dtype if grad is None else grad.dtype)),
           "tt_emb_dense_set_table")


def tt_emb_dense_workspace_size(h, max_tokens: int) -> int:
    out = ctypes.c_size_t()
    _check(lib().tt_emb_dense_workspace_size(h, int(max_tokens), ctypes.byref(out)), "tt_emb_dense_workspace_size")
    return int(out.value)


def tt_emb_dense_set_workspace(h, workspace, max_tokens: int):
    ptr = _dev_ptr(workspace, torch.uint8, "workspace")
    _check(lib().tt_emb_dense_set_workspace(h, ptr, workspace.numel(), int(max_tokens)),
           "tt_emb_dense_set_workspace")


def tt_emb_dense_forward(h, tokens, out, dim: int, stream=None):
    ptr, nbytes, n = _tokens(tokens)
    optr, otype, stride = _rows(out, n, dim, "out")
    rc = lib().tt_emb_dense_forward(h, ptr, nbytes, n, optr, otype, stride, _stream_on(stream, tokens.get_device()))
    if rc:
        raise TTEmbError(rc, "tt_emb_dense_forward")


def tt_emb_dense_backward(h, tokens, grad_out, dim: int, accumulate: bool = False, stream=None):
    ptr, nbytes, n = _tokens(tokens)
    gptr, gtype, stride = _rows(grad_out, n, dim, "grad_out")
    rc = lib().tt_emb_dense_backward(h, ptr, nbytes, n, gptr, gtype, stride, 1 if accumulate else 0,
                                     _stream_on(stream, tokens.get_device()))
    if rc:
        raise TTEmbError(rc, "tt_emb_dense_backward")


def tt_emb_dense_sync(h):
    _check(lib().tt_emb_dense_sync(h), "tt_emb_dense_sync")


def tt_emb_dense_last_error(h) -> int:
    return int(lib().tt_emb_dense_last_error(h))


def tt_emb_dense_destroy(h):
    if h is not None and h.value:
        lib().tt_emb_dense_destroy(h)


def tt_emb_status_word(h) -> int:
    """Device address of a TT handle's status word (0 for a null handle)."""
    return lib().tt_emb_status_word(h) or 0


def tt_emb_dense_status_word(h) -> int:
    return lib().tt_emb_dense_status_word(h) or 0


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
def tt_emb_adamw_create(tensors, options: AdamWOptions, steps):
    """tensors: a list of AdamWTensor; steps: a CUDA int64 tensor of one value."""
    arr = (AdamWTensor * len(tensors))(*tensors)
    h = ctypes.c_void_p()
    _check(lib().tt_emb_adamw_create(len(tensors), arr, ctypes.byref(options),
                                     _dev_ptr(steps, torch.int64, "steps"), ctypes.byref(h)), "tt_emb_adamw_create")
    return h


def tt_emb_adamw_step(h, lr, stream=None):
    """lr: a number, or a CUDA float32 tensor of one value that the device reads."""
    at = None
    if isinstance(lr, torch.Tensor):
        if lr.numel() != 1:
            raise ValueError("lr must have one value")
        at, lr = _dev_ptr(lr, torch.float32, "lr"), 0.0
    rc = lib().tt_emb_adamw_step(h, float(lr), at, _stream_on(stream, torch.cuda.current_device()))
    if rc:
        raise TTEmbError(rc, "tt_emb_adamw_step")


def tt_emb_adamw_destroy(h):
    if h is not None and h.value:
        lib().tt_emb_adamw_destroy(h)
