"""beam_select's order of equal totals, over beams and within one: the whole list."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _expected(scores, groups, beams, k):
    """(beams, ids) by (score, beam, column) where beams differ in nothing else."""
    out = []
    for g in range(groups):
        s = scores[g * beams:(g + 1) * beams]
        b, c = np.divmod(np.arange(s.size), s.shape[1])
        order = np.lexsort((c, b, -s.reshape(-1)))[:k]
        out.append((b[order], c[order]))
    return np.stack([o[0] for o in out]), np.stack([o[1] for o in out])


@pytest.mark.parametrize("name", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("groups,beams,cols,k", [
    (2, 4, 4001, 10), (2, 4, 4000, 100), (1, 8, 64, 40), (3, 16, 33, 128), (1, 3, 70_000, 33)])
@pytest.mark.parametrize("repeated", [True, False])
def test_beams_that_share_a_row(name, groups, beams, cols, k, repeated):
    """One row for all (by a stride of 0, or copied): every score is in the list as often as
    there are beams, and more often where a row has equal ones."""
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    r = np.random.default_rng(cols + k)
    row = torch.from_numpy((r.standard_normal((1, cols)) * 3).astype(np.float32)).to(
        getattr(torch, name)).cuda()
    s = row.expand(groups * beams, cols)
    if not repeated:
        s = s.contiguous()
    t = torch.full((groups, beams), -1.5, device="cuda")
    totals, which, ids = B.beam_select(s, t, k)
    b, c = _expected(s.double().cpu().numpy(), groups, beams, k)
    assert np.array_equal(which.cpu().numpy(), b) and np.array_equal(ids.cpu().numpy(), c)
    assert (totals[:, 1:] <= totals[:, :-1]).all()
