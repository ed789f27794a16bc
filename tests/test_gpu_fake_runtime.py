"""What dense tables do where the CUDA runtime answers otherwise than on one whole GPU: a small library in front of
the runtime, in a process of its own, changes its answers (no second GPU and no part of a GPU is needed)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    out = tmp_path_factory.mktemp("fake") / "libfake.so"
    subprocess.run(["gcc", "-O1", "-fPIC", "-shared", "-I/usr/local/cuda/include", os.path.join(HERE, "fake_cudart.c"), "-o", str(out), "-ldl"],
                   check=True)
    return str(out)


def _run(fake, program):
    env = dict(os.environ, LD_PRELOAD=fake, PYTHONPATH=os.pathsep.join([os.path.dirname(HERE), HERE, os.environ.get("PYTHONPATH", "")]))
    p = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=600, env=env)
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-4000:]


OTHER_DEVICE = """
import ctypes
import torch
from tensor_train_compressed_mixed_b200 import DenseEmbedding, abi
fake = ctypes.CDLL(None)
e = DenseEmbedding(30, 8)
e.set_table(torch.zeros(30, 8, device="cuda"))
bad = torch.tensor([1, 30, 2], device="cuda")
e.forward(bad)
torch.cuda.synchronize()
for stream in (None, 1):
    if stream:                          # a call whose stream is not the device's own
        e.forward(bad, stream=torch.cuda.Stream())
        torch.cuda.synchronize()
    fake.fake_device(1)
    codes = [abi.lib().tt_emb_dense_sync(e.handle) for _ in range(2)]
    fake.fake_device(-1)
    assert codes == [abi.TT_ERR_STATE] * 2, codes
    assert abi.tt_emb_dense_last_error(e.handle) == abi.TT_ERR_STATE
    assert abi.lib().tt_emb_dense_sync(e.handle) == abi.TT_ERR_INDEX_RANGE      # the error was not lost
    assert abi.lib().tt_emb_dense_sync(e.handle) == abi.TT_OK
"""


def test_sync_with_another_device_current_reads_nothing(fake):
    _run(fake, OTHER_DEVICE)


NO_CLUSTERS = """
import ctypes
import torch
from tensor_train_compressed_mixed_b200 import DenseEmbedding, abi
from test_gpu_dense import LAWS, _check_grad
fake = ctypes.CDLL(None)
for n, rows, dim, accumulate, pad in ((257, 40, 8, False, None), (5000, 1, 24, True, None), (5000, 300, 515, False, 7), (40000, 70001, 16, True, 9),
                                      (131072, 3001, 40, False, 0)):
    for law in ("uniform", "runs"):
        g = torch.Generator().manual_seed(n)
        tok, up = LAWS[law](n, rows, g).cuda(), torch.randn(n, dim, generator=g).cuda()
        start = torch.randn(rows, dim, generator=g).cuda()
        sums = []
        for none_fits in (1, 0):
            fake.fake_no_clusters(none_fits)
            launches = fake.fake_cluster_launches()
            e = DenseEmbedding(rows, dim, scale=0.7, padding_idx=pad)
            e.set_table(start, grad=start.clone())
            e.backward(tok, up, accumulate=accumulate)
            e.sync()
            _check_grad(e, tok, up, start.double().cpu() if accumulate else None, 0.7, pad, torch.float32)
            assert fake.fake_cluster_launches() - launches == 1 - none_fits
            sums.append(e.grad)
        assert torch.equal(sums[0], sums[1])        # the order of the sums is that of the sorted tokens, however sorted
"""


def test_gradient_where_no_cluster_of_sixteen_fits(fake):
    _run(fake, NO_CLUSTERS)
