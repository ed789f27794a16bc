"""The projection's workspaces: how much they hold, and that none is given up while a call or a graph still uses it."""
import pytest
import torch

from tensor_train_compressed_mixed_b200 import DenseEmbedding, abi
from test_gpu_project import BF16, F32, _randn, _table

pytestmark = pytest.mark.gpu


def _need(e, x):
    out = torch.empty(*x.shape[:-1], e.num_rows, dtype=e.dtype, device="cuda")
    return abi.tt_emb_dense_project_workspace_size(e.handle, abi.project_call(x, e.num_rows, e.dim, out))


@pytest.mark.parametrize("other", ["current", "another", "a handle"])
def test_growing_batches_keep_one_workspace(other):
    g = torch.Generator(device="cuda").manual_seed(1)
    e, w = _table(2000, 512, F32, g)
    x = _randn(g, 8192, 512)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    keep = torch.cuda.Stream()
    side = {"current": None, "another": keep, "a handle": keep.cuda_stream}[other]
    n = 64
    while n < 8192:
        e.project(x[:n], stream=side)
        n = n * 5 // 4
    torch.cuda.synchronize()
    need = _need(e, x[:n * 4 // 5])
    assert need > 20 << 20
    torch.empty(1, device="cuda")        # blocks that waited for another stream are taken back at the next allocation
    assert torch.cuda.memory_allocated() - before <= 1.5 * need + (1 << 20)
    e.sync()


def _fill(nbytes):
    """Memory that is free to the current stream, overwritten."""
    return [torch.full((nbytes // k,), 0xff, dtype=torch.uint8, device="cuda") for k in (1, 1, 2, 2, 4)]


@pytest.mark.parametrize("kind", [F32, BF16])
def test_a_graph_keeps_its_workspace(kind):
    """bf16 rows at odd places are copied to the workspace, too."""
    g = torch.Generator(device="cuda").manual_seed(2)
    rows, dim, n = 1000, 257, 200
    e, w = _table(rows, dim, kind, g)
    x, y = _randn(g, n, dim, dtype=kind), torch.empty(n, rows, device="cuda")
    e.project(x, out=y)
    want = y.clone()
    graphs = []
    for k in range(2):                   # two graphs of one workspace, and between them a larger one
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            e.project(x, out=y)
        graphs.append(graph)
        big = _randn(g, 3000 * (k + 1), dim, dtype=kind)
        need = _need(e, x)
        e.project(big)
        held = _fill(need)
        for graph in graphs:
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
        assert all((t == 0xff).all() for t in held)
        del held
    e.project(x, out=y)
    e.sync()
    assert torch.equal(y, want)


def test_a_workspace_lives_until_the_calls_on_another_stream_have_ended():
    g = torch.Generator(device="cuda").manual_seed(3)
    rows, dim, n = 1000, 256, 500
    e, w = _table(rows, dim, F32, g)
    x, big = _randn(g, n, dim), _randn(g, 4 * n, dim)
    want = e.project(x)                                   # the workspace is the current stream's
    y = torch.empty_like(want)
    torch.cuda.synchronize()
    first, second = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(first):
        torch.cuda._sleep(200_000_000)                    # some 0.1 s
        e.project(x, out=y)
    second.wait_stream(first)                             # ordered, as one object's calls are
    e.project(big, stream=second)                         # a larger one takes its place
    held = _fill(_need(e, x))                             # the current stream waits for nobody
    torch.cuda.synchronize()
    assert torch.equal(y, want) and all((t == 0xff).all() for t in held)
    e.sync()
