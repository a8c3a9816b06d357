"""topk_distill with lists that are masked throughout by the type's lowest value."""

import numpy as np
import pytest

import scores_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols,k", [(300, 7), (40_000, 50)])
@pytest.mark.parametrize("tau", [0.25, 0.5, 1.0])
def test_every_listed_column_at_the_lowest_value(dtype, cols, k, tau):
    """The loss is tau times the mean distance of the listed scores from the row's
    maximum, about the type's largest value, and finite for tau <= 1 unless it passes
    fp32 itself. Sums of k products, each rounded, of weights that err by 2^-20."""
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    rows = 64
    r = np.random.default_rng(k)
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    low = torch.finfo(dt).min
    tv = np.sort(r.standard_normal((rows, k)).astype(np.float32) * 2, axis=1)
    ti = np.stack([r.permutation(cols)[:k] for _ in range(rows)]).astype(np.int64)
    s = torch.from_numpy((r.standard_normal((rows, cols)) * 3).astype(np.float32)).to(dt)
    s.scatter_(1, torch.from_numpy(ti), low)
    s = s.cuda()
    tvd, tid = torch.from_numpy(tv).cuda(), torch.from_numpy(ti).cuda()
    g = torch.ones(rows, device="cuda")
    forward, stats = B.topk_distill_forward(s, tvd, tid, tau, negated=True)
    both, grad = B.topk_distill(s, tvd, tid, g, tau, negated=True)
    assert torch.equal(grad, B.topk_distill_backward(s, tvd, tid, stats, g, tau, negated=True))
    want = R.distill(s.double().cpu().numpy(), tv, ti, tau, True)[0]
    top, err = float(np.finfo(np.float32).max), k * 2.0 ** -24 + 2.0 ** -20
    for loss in (forward, both):
        loss = loss.double().cpu().numpy()
        fin = np.isfinite(loss)
        assert (np.abs(loss[fin] - want[fin]) <= err * want[fin]).all()
        assert (want[~fin] * (1 + err) > top).all() and not np.isnan(loss).any()
    assert bool(torch.isfinite(grad.float()).all())
