"""What the table's projection, the global norm and the clipped step refuse on the host, before any device work: in a
process whose CUDA runtime is a stand-in that makes handles and refuses launches."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from tensor_train_compressed_mixed_b200 import GradNorm, abi

HERE = os.path.dirname(os.path.abspath(__file__))
MB = 1 << 20
INF, NAN = float("inf"), float("nan")


class Project(ctypes.Structure):
    _fields_ = ([(k, ctypes.c_void_p) for k in ("x", "bias", "residual", "pre", "out")]
                + [(k, ctypes.c_int64) for k in ("x_stride", "residual_stride", "pre_stride", "out_stride", "n")]
                + [(k, ctypes.c_int32) for k in ("bias_type", "residual_type", "pre_type", "out_type", "activation")]
                + [("cap", ctypes.c_float)])


class ProjectGrad(ctypes.Structure):
    _fields_ = ([(k, ctypes.c_void_p) for k in ("x", "grad_out", "pre", "grad_x", "grad_bias")]
                + [(k, ctypes.c_int64) for k in ("x_stride", "grad_out_stride", "pre_stride", "grad_x_stride", "n")]
                + [(k, ctypes.c_int32) for k in ("grad_out_type", "pre_type", "grad_x_type", "grad_bias_type", "activation")]
                + [("cap", ctypes.c_float), ("table_grad", ctypes.c_int32), ("accumulate", ctypes.c_int32)])


def test_calls_are_packed_as_the_header_lays_them_out():
    assert ctypes.sizeof(Project) == abi._PROJECT.size == 104
    assert ctypes.sizeof(ProjectGrad) == abi._PROJECT_GRAD.size == 112
    p = Project.from_buffer_copy(abi._PROJECT.pack(1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16.0))
    assert [getattr(p, k) for k, _ in Project._fields_] == [*range(1, 16), 16.0]
    g = ProjectGrad.from_buffer_copy(abi._PROJECT_GRAD.pack(1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16.0, 17, 18))
    assert [getattr(g, k) for k, _ in ProjectGrad._fields_] == [*range(1, 16), 16.0, 17, 18]


# a table of 10 rows of 6 fp32 values and a call of 4 rows, each buffer at a place of its own
FORWARD = dict(x=1 * MB, bias=2 * MB, residual=3 * MB, pre=4 * MB, out=5 * MB, x_stride=6, residual_stride=10, pre_stride=10, out_stride=10,
               n=4, activation=abi.TT_ACT_GELU)
BACKWARD = dict(x=1 * MB, grad_out=2 * MB, pre=3 * MB, grad_x=4 * MB, grad_bias=5 * MB, x_stride=6, grad_out_stride=10, pre_stride=10,
                grad_x_stride=6, n=4, activation=abi.TT_ACT_GELU, table_grad=1)
TABLE, GRAD = 8 * MB, 9 * MB

BAD_FORWARD = [
    dict(n=-1), dict(n=2 ** 31 - 1), dict(x=None), dict(out=None), dict(x=1 * MB + 2), dict(out=5 * MB + 1), dict(x_stride=-1),
    dict(out_stride=9), dict(pre_stride=9), dict(residual_stride=-1), dict(out_type=3), dict(pre_type=-1), dict(bias_type=3),
    dict(residual_type=7), dict(bias=2 * MB + 2), dict(activation=5), dict(activation=-1),
    dict(activation=abi.TT_ACT_SOFTCAP, cap=0.0), dict(activation=abi.TT_ACT_SOFTCAP, cap=-1.0),
    dict(activation=abi.TT_ACT_SOFTCAP, cap=NAN), dict(activation=abi.TT_ACT_SOFTCAP, cap=INF),
    # outputs on another buffer
    dict(out=1 * MB), dict(out=TABLE), dict(out=TABLE + 236), dict(out=2 * MB), dict(out=4 * MB), dict(pre=1 * MB + 92), dict(pre=TABLE), dict(pre=3 * MB),
    dict(pre=2 * MB - 156), dict(out=3 * MB + 4), dict(out=3 * MB, out_type=abi.TT_BF16), dict(out=3 * MB, residual_stride=11),
    dict(out=4 * MB + 40, out_stride=20, pre_stride=15),
    dict(out=4 * MB + 40, out_stride=19, pre_stride=19), dict(out=4 * MB + 36, out_stride=20, pre_stride=20),
]
GOOD_FORWARD = [
    {}, dict(n=0), dict(bias=None), dict(pre=None), dict(residual=None), dict(x_stride=0), dict(residual_stride=0), dict(x_stride=3),
    dict(out=3 * MB), dict(out=TABLE + 240), dict(pre=2 * MB + 40), dict(activation=abi.TT_ACT_SOFTCAP, cap=30.0),
    # parts of one wider buffer
    dict(out=4 * MB + 40, out_stride=20, pre_stride=20), dict(out=4 * MB - 40, out_stride=20, pre_stride=20),
]
BAD_BACKWARD = [
    dict(n=-1), dict(n=2 ** 31 - 1), dict(x=None), dict(grad_out=None), dict(pre=None), dict(grad_out=2 * MB + 2), dict(grad_x_stride=5),
    dict(grad_out_stride=-1), dict(x_stride=-1), dict(grad_out_type=3), dict(pre_type=3), dict(grad_x_type=3), dict(grad_bias_type=9),
    dict(grad_bias=5 * MB + 2), dict(activation=9), dict(activation=abi.TT_ACT_SOFTCAP, cap=0.0), dict(table_grad=2), dict(accumulate=2),
    dict(grad_x=1 * MB), dict(grad_x=2 * MB + 4), dict(grad_x=TABLE), dict(grad_x=GRAD), dict(grad_x=5 * MB), dict(grad_bias=TABLE + 200),
    dict(grad_bias=GRAD), dict(grad_out=GRAD), dict(x=GRAD + 100), dict(pre=GRAD), dict(grad_bias=3 * MB),
]
GOOD_BACKWARD = [
    {}, dict(n=0), dict(x=None, table_grad=0), dict(grad_x=None), dict(grad_bias=None), dict(pre=None, activation=0), dict(grad_out_stride=0),
    dict(accumulate=1), dict(x_stride=0), dict(pre=2 * MB), dict(grad_x=GRAD, table_grad=0),
]

PROGRAM = """
import ctypes, sys
sys.path[:0] = [{root!r}, {here!r}]
import test_project_cpu as t
t.inside()
"""


def _handle(L, kind=abi.TT_F32, grad=GRAD):
    h = ctypes.c_void_p()
    assert L.tt_emb_dense_create(10, 6, kind, 1.0, -1, ctypes.byref(h)) == abi.TT_OK
    assert L.tt_emb_dense_set_table(h, TABLE, grad, abi.TT_F32) == abi.TT_OK
    return h


def inside():
    """Runs in the process with the stand-in runtime."""
    L = abi.lib()
    size = ctypes.c_size_t()
    calls = [(Project, FORWARD, L.tt_emb_dense_project, L.tt_emb_dense_project_workspace_size, BAD_FORWARD, GOOD_FORWARD),
             (ProjectGrad, BACKWARD, L.tt_emb_dense_project_backward, L.tt_emb_dense_project_backward_workspace_size, BAD_BACKWARD, GOOD_BACKWARD)]
    for kind, base, call, sized, bad, good in calls:
        h = _handle(L)
        for kw in bad:
            c = bytes(kind(**{**base, **kw}))
            assert sized(h, c, ctypes.byref(size)) == abi.TT_ERR_ARG, kw
            assert call(h, c, None) == abi.TT_ERR_ARG, kw
            assert L.tt_emb_dense_last_error(h) == abi.TT_ERR_ARG
        for kw in good:
            c = bytes(kind(**{**base, **kw}))
            assert sized(h, c, ctypes.byref(size)) == abi.TT_OK, kw
            rc = call(h, c, None)           # up to the workspace, or the launch that the stand-in refuses
            assert rc in (abi.TT_ERR_WORKSPACE, abi.TT_ERR_CUDA) or (kw.get("n") == 0 and rc == abi.TT_OK), (kw, rc)
        c = bytes(kind(**base))
        assert sized(h, c, None) == sized(h, None, ctypes.byref(size)) == call(h, None, None) == call(None, c, None) == abi.TT_ERR_ARG
        assert L.tt_emb_dense_set_project_workspace(h, None, 0) == L.tt_emb_dense_set_project_workspace(h, MB + 8, MB) == abi.TT_ERR_ARG
        assert L.tt_emb_dense_set_project_workspace(None, MB, MB) == abi.TT_ERR_ARG
        bare = ctypes.c_void_p()
        assert L.tt_emb_dense_create(10, 6, abi.TT_F32, 1.0, -1, ctypes.byref(bare)) == abi.TT_OK
        assert call(bare, c, None) == abi.TT_ERR_STATE
    h = _handle(L, grad=None)
    assert L.tt_emb_dense_project_backward(h, bytes(ProjectGrad(**BACKWARD)), None) == abi.TT_ERR_STATE
    _norms(L)


def _norms(L):
    def make(*recs):
        h = ctypes.c_void_p(1)
        rc = L.tt_emb_norm_create(len(recs), (abi.NormTensor * max(1, len(recs)))(*recs), ctypes.byref(h))
        assert (rc == abi.TT_OK) == bool(h.value)
        return rc, h

    def rec(**kw):
        return abi.NormTensor(**{**dict(grad=1 * MB, size=100, grad_type=abi.TT_F32), **kw})

    for kw in (dict(size=-1), dict(size=2 ** 41), dict(grad=None), dict(grad=MB + 2), dict(grad_type=3), dict(guard=MB + 2), dict(reserved=1)):
        assert make(rec(**kw))[0] == abi.TT_ERR_ARG, kw
    assert make()[0] == abi.TT_ERR_ARG
    assert L.tt_emb_norm_create(1, None, ctypes.byref(ctypes.c_void_p())) == L.tt_emb_norm_create(1, (abi.NormTensor * 1)(rec()), None) == abi.TT_ERR_ARG
    rc, h = make(rec(), rec(grad=2 * MB, grad_type=abi.TT_BF16), rec(size=0, grad=None))
    assert rc == abi.TT_OK
    for bound in (0.0, -1.0, NAN):
        assert L.tt_emb_norm_clip(h, bound, 4 * MB, None) == abi.TT_ERR_ARG
    for at in (4 * MB + 2, MB, MB + 396, 2 * MB + 196):
        assert L.tt_emb_norm_clip(h, 1.0, at, None) == L.tt_emb_norm_measure(h, at, None) == abi.TT_ERR_ARG, at
    assert L.tt_emb_norm_measure(h, None, None) == abi.TT_ERR_ARG
    assert L.tt_emb_norm_clip(h, INF, MB + 400, None) == abi.TT_ERR_CUDA       # accepted up to the launch
    rc, h = make(rec(), rec(grad=MB + 396))
    assert rc == abi.TT_OK
    assert L.tt_emb_norm_clip(h, 1.0, 4 * MB, None) == abi.TT_ERR_ARG           # one value would be scaled twice
    assert L.tt_emb_norm_measure(h, 4 * MB, None) == abi.TT_ERR_CUDA
    t = abi.AdamWTensor(param=MB, grad=2 * MB, exp_avg=3 * MB, exp_avg_sq=4 * MB, size=100)
    o = abi.AdamWOptions(beta1=0.9, beta2=0.999, eps=1e-8, state_bits=32)
    h = ctypes.c_void_p()
    assert L.tt_emb_adamw_create(1, (abi.AdamWTensor * 1)(t), ctypes.byref(o), 5 * MB, ctypes.byref(h)) == abi.TT_OK
    for bound in (0.0, -1.0, NAN):
        assert L.tt_emb_adamw_step_clipped(h, 0.1, None, bound, None, None) == abi.TT_ERR_ARG
    for at in (MB, 2 * MB + 396, 3 * MB - 0, 4 * MB + 8, 5 * MB + 4, 6 * MB, 6 * MB + 2):
        assert L.tt_emb_adamw_step_clipped(h, 0.1, 6 * MB, 1.0, at, None) == abi.TT_ERR_ARG, at
    assert L.tt_emb_adamw_step_clipped(h, -0.1, None, 1.0, None, None) == abi.TT_ERR_ARG
    assert L.tt_emb_adamw_step_clipped(h, 0.1, None, INF, 7 * MB, None) == abi.TT_ERR_CUDA
    L.tt_emb_adamw_destroy(h)


def test_refusals_on_the_host(tmp_path):
    so = tmp_path / "libhost.so"
    subprocess.run(["gcc", "-O1", "-fPIC", "-shared", "-I/usr/local/cuda/include", os.path.join(HERE, "host_cudart.c"), "-o", str(so)], check=True)
    env = dict(os.environ, LD_PRELOAD=str(so))
    p = subprocess.run([sys.executable, "-c", PROGRAM.format(root=os.path.dirname(HERE), here=HERE)], capture_output=True, text=True, timeout=600, env=env)
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-4000:]


def test_null_handles():
    L = abi.lib()
    assert L.tt_emb_norm_measure(None, MB, None) == L.tt_emb_norm_clip(None, 1.0, MB, None) == abi.TT_ERR_ARG
    assert L.tt_emb_adamw_step_clipped(None, 0.1, None, 1.0, None, None) == abi.TT_ERR_ARG
    L.tt_emb_norm_destroy(None)


def test_python_refuses_what_it_cannot_pass_on():
    x = torch.zeros(4, 6)
    with pytest.raises(TypeError):
        abi.project_call(x, 10, 6, torch.zeros(4, 10))
    for bad in (dict(activation="tanh"), dict(activation="softcap"), dict(cap=3.0), dict(activation="relu", cap=3.0)):
        with pytest.raises(ValueError):
            abi.project_call(x, 10, 6, torch.zeros(4, 10), **bad)
    with pytest.raises(ValueError):
        abi.project_grad_call(x, 10, 6, torch.zeros(4, 10), activation="relu")
    with pytest.raises(ValueError):
        GradNorm([])
    with pytest.raises(ValueError):
        GradNorm([x], guards=[])
    with pytest.raises(TypeError):
        GradNorm([x])
    with pytest.raises(ValueError):
        GradNorm.for_tables([])
    with pytest.raises(TypeError):
        abi._one(torch.zeros(1))
    with pytest.raises(ValueError):
        abi._one(torch.zeros(2))
