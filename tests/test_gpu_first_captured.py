"""The first projection, its gradients and the first clipped step of a process, captured without a call before them."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

PROGRAM = """
import torch
from tensor_train_compressed_mixed_b200 import AdamW, DenseEmbedding, GradNorm
g = torch.Generator(device="cuda").manual_seed(1)
rand = lambda *s, t=torch.float32: torch.randn(*s, generator=g, device="cuda").to(t)
n, rows, dim = 300, 700, 256
w, x, dy, pre = rand(rows, dim, t=KIND), rand(n, dim, t=KIND), rand(n, rows, t=KIND), rand(n, rows, t=KIND)
e = DenseEmbedding(rows, dim, dtype=KIND)
e.set_table(w, grad=torch.zeros(rows, dim, device="cuda"))
a, c = AdamW([w], [e.grad]), GradNorm([e.grad])
w0 = w.clone()

def calls():
    y = e.project(x, activation="gelu")
    gx = e.project_backward(x, dy, pre=pre, activation="gelu")
    c.clip(1.0)
    a.step(0.01, max_norm=0.5)
    return y, gx, e.grad, w
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
w.copy_(w0)
a.steps.zero_(), a.m.zero_(), a.v.zero_()
want = calls()
e.sync()
assert all(torch.equal(p, q) for p, q in zip(got, want)) and not torch.equal(w, w0)
"""


@pytest.mark.parametrize("kind", ["torch.bfloat16", "torch.float32"])
def test_first_calls_captured(kind):
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(HERE), os.environ.get("PYTHONPATH", "")]))
    p = subprocess.run([sys.executable, "-c", PROGRAM.replace("KIND", kind)], capture_output=True, text=True, timeout=600, env=env)
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-4000:]
