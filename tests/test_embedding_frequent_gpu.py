"""embedding_gradient where one token has most of many positions, or few far from each other."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from approximate_nearest_neighbour_gb300 import binding
    return binding


def _check(B, ids, rows, cols=3):
    """Whole numbers below 2^24 in sum: exact. Random values: the same bits each time, so the
    positions are taken in one order."""
    import torch
    n = ids.numel()
    g = torch.randint(-1, 2, (n, cols), device="cuda").float()
    ok = (ids >= 0) & (ids < rows)
    want = torch.zeros((rows, cols), dtype=torch.float64, device="cuda")
    want.index_add_(0, ids[ok].long(), g[ok].double())
    assert torch.equal(B.embedding_gradient(g, ids, rows).double(), want)
    g = torch.randn((n, cols), device="cuda")
    first = B.embedding_gradient(g, ids, rows)
    for _ in range(3):
        assert torch.equal(B.embedding_gradient(g, ids, rows), first)


@pytest.mark.parametrize("wide", [False, True])
def test_most_positions_are_of_one_token(B, wide):
    import torch
    r = np.random.default_rng(1)
    n = 1 << 20
    for share, rows in ((1.0, 10), (0.5, 1000), (0.1, 300), (0.02, 5000)):
        ids = np.where(r.random(n) < share, 7, r.integers(-1, rows, n))
        _check(B, torch.from_numpy(ids if wide else ids.astype(np.int32)).cuda(), rows)


def test_positions_in_few_ranges(B):
    """A token's positions at both ends and in between, with ranges that hold none."""
    import torch
    n = (1 << 21) + 77
    for count in (129, 3000, 20_000):  # by a bitmap; in shared memory and not
        ids = torch.full((n,), -1, dtype=torch.int32, device="cuda")
        for first in (0, 32_768 * 9 - count // 6, 1_000_000, n - count // 3):
            ids[first:first + count // 3] = 5
        ids[1_500_000:1_500_000 + count * 3:3] = 133  # the same class
        _check(B, ids, 200)


def test_time_grows_with_the_positions(B):
    """Four times the positions of one token take four times as long, and no sixteen."""
    import torch
    took = []
    for n in (1 << 21, 1 << 23):
        ids = torch.full((n,), 3, dtype=torch.int32, device="cuda")
        g = torch.ones((n, 1), device="cuda")
        best = float("inf")
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            got = B.embedding_gradient(g, ids, 8)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        assert got[3, 0] == n
        took.append(best)
    assert took[1] < 8 * took[0], took
