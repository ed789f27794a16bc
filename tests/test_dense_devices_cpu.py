"""The library's calls of a DenseEmbedding run with the table's own device current, whichever one the caller left current."""
import contextlib

import pytest
import torch

from tensor_train_compressed_mixed_b200 import abi, dense


@pytest.fixture
def second(monkeypatch):
    """A table on the second device, the first being current, over a library that notes the current device."""
    current, calls = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    for name in ("create", "sync", "destroy", "forward", "backward"):
        monkeypatch.setattr(abi, f"tt_emb_dense_{name}", lambda *a, name=name: calls.append((name, current[0])))
    e = dense.DenseEmbedding(10, 4, device="cuda:1")
    e._ws_tokens = 100
    monkeypatch.setattr(e, "_check", lambda *a: None)
    yield e, calls
    assert current == [0]
    e.handle = None


def test_calls_run_on_the_tables_device(second):
    e, calls = second
    tok = torch.zeros(3, dtype=torch.int64)
    e.forward(tok, out=torch.zeros(3, 4))
    e.backward(tok, torch.zeros(3, 4))
    e.sync()
    assert calls == [(name, 1) for name in ("create", "forward", "backward", "sync")]
