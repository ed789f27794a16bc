"""What making a handle asks of the CUDA runtime: one allocation and one wait, and nothing for calls that may never come; what its test hook refuses."""
import ctypes
import os
import subprocess
import sys

from tensor_train_compressed_mixed_b200 import abi

HERE = os.path.dirname(os.path.abspath(__file__))
MB = 1 << 20

PROGRAM = """
import sys
sys.path[:0] = [{root!r}, {here!r}]
import test_creation_cpu as t
t.{what}()
"""


def _taken():
    n = (ctypes.c_int * 3)()
    ctypes.CDLL(None).count_take(n)
    return list(n)


def _run(tmp_path, what):
    so = tmp_path / "libcount.so"
    subprocess.run(["gcc", "-O1", "-fPIC", "-shared", "-I/usr/local/cuda/include", os.path.join(HERE, "count_cudart.c"), "-o", str(so)], check=True)
    p = subprocess.run([sys.executable, "-c", PROGRAM.format(root=os.path.dirname(HERE), here=HERE, what=what)], capture_output=True, text=True, timeout=600,
                       env=dict(os.environ, LD_PRELOAD=str(so)))
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-4000:]


def adamw():
    L = abi.lib()
    t = abi.AdamWTensor(param=MB, grad=2 * MB, exp_avg=3 * MB, exp_avg_sq=4 * MB, size=100)
    o = abi.AdamWOptions(beta1=0.9, beta2=0.999, eps=1e-8, state_bits=32)
    h = ctypes.c_void_p()
    _taken()
    assert L.tt_emb_adamw_create(1, (abi.AdamWTensor * 1)(t), ctypes.byref(o), 5 * MB, ctypes.byref(h)) == abi.TT_OK
    assert _taken() == [1, 1, 0]
    assert L.tt_emb_adamw_step_clipped(h, 0.1, None, 1.0, None, None) == abi.TT_ERR_CUDA      # up to the launch
    assert _taken() == [0, 0, 0]
    L.tt_emb_adamw_destroy(h)


def norm():
    L = abi.lib()
    h = ctypes.c_void_p()
    _taken()
    assert L.tt_emb_norm_create(1, (abi.NormTensor * 1)(abi.NormTensor(grad=MB, size=100, grad_type=abi.TT_F32)), ctypes.byref(h)) == abi.TT_OK
    assert _taken() == [1, 1, 1]
    L.tt_emb_norm_destroy(h)


def test_adamw(tmp_path):
    _run(tmp_path, "adamw")


def test_norm(tmp_path):
    _run(tmp_path, "norm")


def dense():
    from test_project_cpu import FORWARD, Project, _handle
    L = abi.lib()
    h = ctypes.c_void_p()
    _taken()
    assert L.tt_emb_dense_create(10, 6, abi.TT_F32, 1.0, -1, ctypes.byref(h)) == abi.TT_OK
    assert _taken() == [1, 1, 5]                     # of the kernels that sort tokens
    L.tt_emb_dense_destroy(h)
    h = _handle(L, abi.TT_BF16)
    _taken()
    size, call = ctypes.c_size_t(), bytes(Project(**FORWARD))
    for asked in (0, 0):                             # a product this small has no plan
        assert L.tt_emb_dense_project_workspace_size(h, call, ctypes.byref(size)) == abi.TT_OK and size.value == 0
        assert _taken() == [0, 0, asked]
    L.tt_emb_dense_destroy(h)
    assert L.tt_emb_dense_create(1000, 512, abi.TT_F32, 1.0, -1, ctypes.byref(h)) == abi.TT_OK
    assert L.tt_emb_dense_set_table(h, 8 * MB, None, abi.TT_F32) == abi.TT_OK
    _taken()
    call = bytes(Project(**{**FORWARD, "x_stride": 512, "residual_stride": 1000, "pre_stride": 1000, "out_stride": 1000}))
    for asked in (6, 0):                             # the product kernels', once
        assert L.tt_emb_dense_project_workspace_size(h, call, ctypes.byref(size)) == abi.TT_OK and size.value > 0
        assert _taken() == [0, 0, asked]


def test_dense(tmp_path):
    _run(tmp_path, "dense")


def hook():
    from test_project_cpu import _handle
    L = abi.lib()
    h = _handle(L)
    for what in (abi.TT_INJECT_COPIES, abi.TT_INJECT_PRODUCTS, abi.TT_INJECT_SUMS, abi.TT_INJECT_NONE):
        assert L.tt_emb_dense_debug_inject(h, what) == abi.TT_OK
    for what in (-1, abi.TT_INJECT_POOL_WAIT, abi.TT_INJECT_MMA_WAIT_BWD, 7):
        assert L.tt_emb_dense_debug_inject(h, what) == abi.TT_ERR_ARG
    assert L.tt_emb_dense_debug_inject(None, abi.TT_INJECT_NONE) == abi.TT_ERR_ARG


def test_hook(tmp_path):
    _run(tmp_path, "hook")
