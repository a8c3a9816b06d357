"""NVFP4 with matrix scales at the ends of fp32."""

import numpy as np
import pytest

import scores_ref as R
from test_fp4_gpu import _check_quantized

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from approximate_nearest_neighbour_gb300 import binding
    return binding


def _round_trip(B, x, g):
    import torch
    t, gt = torch.from_numpy(x).cuda(), torch.tensor([g], device="cuda")
    assert float(gt) == g
    codes, scales = B.fp4_quantize(t, "nvfp4", tensor_scale=gt)
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    _check_quantized(x.astype(np.float64), c, s, "nvfp4", gt)
    want = torch.from_numpy((R.values(c, s, "nvfp4") * g).astype(np.float32))
    got = B.fp4_dequantize(codes, scales, x.shape[1], "nvfp4", tensor_scale=gt).cpu()
    assert torch.equal(got, want)
    assert bool((got != 0).any())


@pytest.mark.parametrize("e", [-110, -118, -122, -126, -130, -134, -140])
@pytest.mark.parametrize("mantissa", [1.0, 1.4375])
def test_small_scales(B, e, mantissa):
    """Blocks whose scale times the matrix's is subnormal: its reciprocal passes fp32."""
    r = np.random.default_rng(-e)
    g = mantissa * 2.0 ** e
    # block maxima from E4M3's smallest scales to its largest, and past it
    top = 6 * g * 2.0 ** r.uniform(-8, 10, (64, 8, 1))
    x = (top * r.uniform(-1, 1, (64, 8, 16))).reshape(64, 128).astype(np.float32)
    x[0, :16] = 0
    _round_trip(B, x, g)
    x[5, 3], x[9, 20] = 1.0, -3e38  # far above what the scale can hold: saturates
    _round_trip(B, x, g)


@pytest.mark.parametrize("g", [2.0 ** 125, 2.0 ** 126, 1.75 * 2.0 ** 126])
def test_large_scales(B, g):
    """Six times the matrix's scale passes fp32."""
    r = np.random.default_rng(7)
    x = (r.uniform(-1, 1, (40, 96)) * 2.0 ** r.uniform(118, 127, (40, 1))).astype(np.float32)
    _round_trip(B, x, g)
