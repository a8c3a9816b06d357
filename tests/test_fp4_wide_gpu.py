"""The product of many packed rows (fp4_wide.cu): every tile shape, CTA pairs, stages
whose rows of a are kept, all output types, and fp4_linear on top, against fp64.

The shapes take the same variant on 148 to 160 SMs.
"""

import numpy as np
import pytest

import scores_ref as R

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]


@pytest.fixture(scope="module")
def B():
    from approximate_nearest_neighbour_gb300 import binding
    return binding


def _dt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _x(rows, cols, seed, dtype="f32"):
    """Normal values whose rows differ in magnitude, with zeros among them."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    x *= 2.0 ** torch.randint(-4, 5, (rows, 1), generator=gen, device="cuda")
    x[torch.rand((rows, cols), generator=gen, device="cuda") < 0.1] = 0
    return x.to(_dt(dtype))


def _g(fmt, v):
    import torch
    return torch.tensor([v], device="cuda") if fmt == "nvfp4" else None


def _values(codes, scales, fmt):
    """What packed rows stand for without the matrix's scale, fp64, from the layout's
    and the formats' definitions."""
    import torch
    rows, pitch = codes.shape
    blk = R.BLOCK[fmt]
    grid = torch.tensor(np.concatenate([R.E2M1, -R.E2M1]), device="cuda")
    v = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).view(rows, -1, blk)
    r = torch.arange(rows, device="cuda")[:, None]
    c = torch.arange(2 * pitch // blk, device="cuda")[None, :]
    s = scales[r // 128, c // 4, (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4]
    byte = np.arange(256 if fmt == "mxfp4" else 128)
    table = torch.tensor(R.scale_value(byte, fmt), device="cuda")
    return (v * table[s.long()][..., None]).view(rows, -1)


def _check(got, va, vb, alpha):
    """As in the small products: fp32 sums of exact terms err by at most cols / 16 + 4
    units of 2^-23 of the sum of magnitudes, whatever the grouping."""
    want = alpha * (va @ vb.T)
    tol = (va.shape[1] / 16 + 4) * 2.0 ** -23 * abs(alpha) * (va.abs() @ vb.abs().T)
    assert bool(((got.double() - want).abs() <= tol).all())


SHAPES = [
    # rows of a x columns of out x K
    (2100, 20000, 96),      # 256-row tiles, short K, several tiles per CTA
    (2111, 20003, 128),     # the same at odd sizes
    (101, 250_001, 128),    # one 128-row tile, a's rows kept in the stages (short K)
    (128, 250_004, 96),
    (200, 250_003, 100),    # one 256-row tile, kept
    (120, 250_002, 300),    # 128-row tile, two stages per tile, kept
    (250, 200_004, 1000),   # 256-row tile, four stages per tile, kept
    (1111, 40_002, 2100),   # pairs of CTAs, the last pair half outside
    (1111, 40_003, 2100),   # odd columns
    (1300, 40_100, 2049),   # the last pair's second half partial, a K step of one column
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,cols", SHAPES)
def test_wide_product(B, fmt, m, n, cols):
    import torch
    ga, gb = _g(fmt, 0.013), _g(fmt, 0.021)
    qa = B.fp4_quantize(_x(m, cols, m), fmt, tensor_scale=ga)
    qb = B.fp4_quantize(_x(n, cols, n), fmt, tensor_scale=gb)
    got = B.fp4_product(*qa, *qb, fmt, a_tensor_scale=ga, b_tensor_scale=gb)
    B.device_check()
    va, vb = _values(*qa, fmt), _values(*qb, fmt)
    alpha = 1.0 if ga is None else float(ga) * float(gb)
    step = max(1, 60_000_000 // n)
    for r in range(0, m, step):
        _check(got[r:r + step], va[r:r + step], vb, alpha)
    for o in ("bf16", "f16"):
        h = B.fp4_product(*qa, *qb, fmt, a_tensor_scale=ga, b_tensor_scale=gb, dtype=_dt(o))
        assert torch.equal(h, got.to(_dt(o)))  # the same sums, rounded once
    again = B.fp4_product(*qa, *qb, fmt, a_tensor_scale=ga, b_tensor_scale=gb)
    B.device_check()
    assert torch.equal(got, again)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,cols",
                         [(300, 20_000, 2100), (700, 20_000, 100), (2500, 20_001, 2100)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_wide_linear(B, fmt, m, n, cols, dtype):
    """128-row tiles, short K, and pairs, started while the rows are still quantized."""
    import torch
    x = _x(m, cols, 3, dtype)
    gx, gw = _g(fmt, 0.05), _g(fmt, 0.03)
    qw = B.fp4_quantize(_x(n, cols, 4), fmt, tensor_scale=gw)
    qx = B.fp4_quantize(x, fmt, tensor_scale=gx)
    want = B.fp4_product(*qx, *qw, fmt, a_tensor_scale=gx, b_tensor_scale=gw)
    _check(want, _values(*qx, fmt), _values(*qw, fmt),
           1.0 if gx is None else float(gx) * float(gw))
    for _ in range(3):
        got = B.fp4_linear(x, *qw, fmt, x_tensor_scale=gx, w_tensor_scale=gw)
        assert got.dtype == x.dtype and torch.equal(got, want.to(x.dtype))
    B.device_check()


@pytest.mark.parametrize("fmt", FMTS)
def test_wide_keeps_rows_apart(B, fmt):
    """A block that is not finite reaches its own row and column of the result only."""
    import torch
    a, b = _x(1200, 2200, 1), _x(40_000, 2200, 2)
    a[3, 100] = float("nan")
    a[1199, 2199] = -float("inf")
    b[39_999, 0] = float("inf")
    out = B.fp4_product(*B.fp4_quantize(a, fmt), *B.fp4_quantize(b, fmt), fmt)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[[3, 1199], :] = True
    want[:, 39_999] = True
    assert torch.equal(torch.isnan(out), want)
