"""score_adjust with temperatures whose reciprocal passes fp32."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from approximate_nearest_neighbour_gb300 import binding
    return binding


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("negate", [False, True])
def test_temperatures_at_the_ends_of_fp32(B, dtype, listed, negate):
    """Scores over temperatures from 2^-149 to 2^127, zero and tiny scores among them.
    Three fp32 roundings (the factor, the product, the scaling back) and a bias that is 0."""
    import torch
    t = np.array([2.0 ** -149, 1e-40, 2.0 ** -128, 2.0 ** -127, 2.0 ** -126, 1e-30, 1, 2.0 ** 127],
                 np.float32)
    r = np.random.default_rng(2)
    x = (r.standard_normal((8, 77)) * 2.0 ** r.uniform(-140, 2, (8, 77))).astype(np.float32)
    x[:, ::5] = 0
    x[:, 3] = np.inf
    x[:, 4] = -np.inf
    x = torch.from_numpy(x).to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
    kw = {}
    if listed:
        kw = {"bias_ids": torch.arange(0, 72, 3, dtype=torch.int32, device="cuda").repeat(8, 1),
              "bias_vals": torch.zeros((8, 24), device="cuda")}
    got = B.score_adjust(x, temperature=torch.from_numpy(t).cuda(), negate=negate,
                         dtype=torch.float32, **kw).cpu().numpy()
    with np.errstate(over="ignore"):
        want = x.double().cpu().numpy() / t.astype(np.float64)[:, None] * (-1 if negate else 1)
        want32 = want.astype(np.float32)
    fin = np.isfinite(want32)
    assert np.array_equal(got[~fin], want32[~fin])
    assert (np.abs(got[fin] - want[fin]) <= 2.0 ** -21 * np.abs(want[fin]) + 2.0 ** -148).all()
