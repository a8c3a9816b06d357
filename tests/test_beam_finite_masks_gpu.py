"""beam_select on scores of any finite size: masks of large finite values, dense ones, and
large scores, against fp64."""

import numpy as np
import pytest

import decode_ref as R

pytestmark = pytest.mark.gpu

# below, at and above 2^30, and towards the end of fp32
FAR = [-1e9, -2.0 ** 30, -2e9, 2e9, -1e10, -1e12, -1e20, -1e30, 1e30, -1e37, -1e38, -3e38]


@pytest.fixture(scope="module")
def B():
    from approximate_nearest_neighbour_gb300 import binding
    return binding


def _rows(cols, far, dtype, seed):
    """Six rows: a hundredth, a thousandth and nothing left beside `far`; one score left
    in the last column; scores of the size of `far` throughout; none masked."""
    import torch
    r = np.random.default_rng(seed)
    s = (r.standard_normal((6, cols)) * 3).astype(np.float32)
    for row, share in ((0, 0.01), (1, 0.001), (2, 0.0)):
        s[row, r.random(cols) >= share] = far
    s[3, :-1] = far
    s[4] = (r.random(cols) * 0.25 + 0.5).astype(np.float32) * np.float32(far)
    return torch.from_numpy(s).to(dtype).cuda()


@pytest.mark.parametrize("name", ["float32", "bfloat16"])
@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("cols", [32_000, 32_001])
def test_far_scores(B, name, far, cols):
    """One kernel (few continuations) and two, whole vectors and rows at odd offsets."""
    import torch
    s = _rows(cols, far, getattr(torch, name), cols)
    scores = s.double().cpu().numpy()
    for groups, k in ((1, 4), (2, 8), (6, 20), (1, 128), (2, 100)):
        t = np.linspace(-3, 0, 6, dtype=np.float32).reshape(groups, 6 // groups)
        got = B.beam_select(s, torch.from_numpy(t).cuda(), k)
        R.check_selection(got, scores, t, k)
        assert (got[1] >= 0).all(), "every row has continuations"


@pytest.mark.parametrize("name", ["float32", "bfloat16"])
def test_far_blocks_of_a_long_row(B, name):
    """Stretches of masked columns, each at its own value, in a row of several blocks."""
    import torch
    r = np.random.default_rng(3)
    s = (r.standard_normal((4, 131_072)) * 3).astype(np.float32)
    for i, far in enumerate(FAR[4:]):
        s[0, i * 16_384:i * 16_384 + 16_000] = -abs(far)
        s[1, i * 16_384 + 300:(i + 1) * 16_384] = -abs(far)
    s[2, 1000:] = -1e30
    s = torch.from_numpy(s).to(getattr(torch, name)).cuda()
    t = np.zeros((2, 2), np.float32)
    for k in (4, 60):
        got = B.beam_select(s, torch.from_numpy(t).cuda(), k)
        R.check_selection(got, s.double().cpu().numpy(), t, k)
