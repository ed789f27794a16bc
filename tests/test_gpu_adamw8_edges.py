"""Edges of the 8-bit moments, code for code against the header's rule: values that are not finite beside
small ones, and blocks whose first moment is near the end of float32's range."""
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


# the last is 0.9 of what float32 ends with, nearly
TOPS = [2.0 ** 124, 2.0 ** 125 * (2 - 2.0 ** -23), 2.0 ** 126, 2.0 ** 126 * (1 + 2.0 ** -23), 1e38, 2.0 ** 126 * (2 - 2.0 ** -23), 2.0 ** 127,
        3.06e38]


@pytest.mark.parametrize("top", TOPS)
def test_first_moments_up_to_the_largest_float(top):
    """The first moment's codes are those of values x (448 x (1 / magnitude)) where 1 / magnitude is below the least
    normal number too.  The second moment is of 1e19, so that weights stay finite."""
    n = 256 * 8
    g = torch.zeros(n, device="cuda")
    p = torch.ones(n, device="cuda")
    o = AdamW([p], [g], betas=(B1, B2), eps=EPS, weight_decay=0.0, state_bits=8, seed=9)
    codes = torch.randint(0x7F, (n,), generator=torch.Generator().manual_seed(5), dtype=torch.uint8)
    codes[::256] = 0x7E                              # 448
    codes[1::2] |= 0x80
    o.m.view(torch.uint8).copy_(codes)
    o.v.view(torch.uint8).fill_(0x7E)
    # the step's 0.9 m is the value wanted or one next to it
    o.m_scale.fill_(top / B1 / 448)
    o.v_scale.fill_(1e19 / 448)
    for t in (1, 2):
        before = _snapshot(o)
        o.step(0.01)
        _check8(o, before, t, float(np.float32(0.01)), 0.0, 9)


def test_a_gradient_that_reaches_the_end_of_the_range_by_itself():
    """Eight steps of 3e38: the moment passes 2^126 at the fourth."""
    n = 512
    g = torch.linspace(-1, 1, n, device="cuda") * 3e38
    p = torch.ones(n, device="cuda")
    o = AdamW([p], [g], betas=(B1, B2), eps=EPS, weight_decay=0.0, state_bits=8, seed=2)
    for t in range(1, 9):
        before = _snapshot(o)
        o.step(0.01)
        _check8(o, before, t, float(np.float32(0.01)), 0.0, 2)
