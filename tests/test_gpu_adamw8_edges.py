"""Edges of the 8-bit moments, code for code against the header's rule: values that are not finite beside small ones."""
import numpy as np
import pytest
import torch

from tensor_train_compressed_mixed_b200 import AdamW
from test_gpu_adamw import B1, B2, EPS, _check8, _snapshot

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), 3e19, -1e30, float("nan")])
def test_small_roots_beside_values_that_are_not_finite(bad, seed):
    """Every group of four values that take one random word holds a value whose square is not finite, at each of
    the four places, and small ones whose roots round to the code zero but for the rule of the least code."""
    n = 256 * 32
    rng = np.random.default_rng(seed)
    g = torch.from_numpy((rng.uniform(0.5, 2.0, n) * 10.0 ** rng.uniform(-9, -6, n)).astype(np.float32)).cuda()
    quad = torch.arange(n // 4, device="cuda")
    g[quad * 4 + quad % 4] = bad
    g[8::256] = 1.0                                 # what the block's scale comes from
    p = torch.zeros(n, device="cuda")
    o = AdamW([p], [g], betas=(B1, B2), eps=EPS, weight_decay=0.0, state_bits=8, seed=seed)
    for t in (1, 2, 3):
        before = _snapshot(o)
        o.step(0.01)
        _check8(o, before, t, float(np.float32(0.01)), 0.0, seed)
    codes = o.v.view(torch.uint8)[torch.isfinite(g) & (g.abs() < 1e18)]
    assert (codes > 0).all()
