"""4-bit block-scaled vectors: quantisation, its inverse, and the products."""

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


def _x(rows, cols, seed, dtype, spread=True):
    """Normal values whose rows and blocks differ widely in magnitude."""
    import torch
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, cols)).astype(np.float32)
    if spread:
        x *= 2.0 ** r.integers(-6, 7, (rows, 1)).astype(np.float32)
        x[r.random((rows, cols)) < 0.1] = 0
    return torch.from_numpy(x).to(_dt(dtype)).cuda()


def _g(fmt, v=0.0371):
    import torch
    return torch.tensor([v], device="cuda") if fmt == "nvfp4" else None


def _check_quantized(x, codes, scales, fmt, g):
    """Scale bytes and codes against the definition. MXFP4 is exact. For NVFP4
    fp32 rounds amax / (6 g) and x * (1 / (s g)) by at most 4 x 2^-24: bytes
    and codes may differ from the fp64 definition only within 2^-21 of a
    rounding boundary."""
    rows = x.shape[0]
    nblk = codes.shape[1] * 2 // R.BLOCK[fmt]
    got = R.untile(scales, rows, nblk)
    gv = 1.0 if g is None else float(g)
    want = R.block_scales(x, fmt, gv)
    b = R.blocks(x, fmt)
    if fmt == "nvfp4":
        v = np.abs(np.where(np.isfinite(b), b, 0)).max(-1) / (6 * gv)
        ok = (got == want) | (R.e4m3_round(v * (1 - 2.0 ** -21)) == got) | \
            (R.e4m3_round(v * (1 + 2.0 ** -21)) == got)
        assert ok.all()
    else:
        assert np.array_equal(got, want)
    s = R.scale_value(got, fmt)[..., None] * gv
    c = R.unpack(codes).reshape(b.shape)
    fin = np.isfinite(s[..., 0])
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s > 0, b / s, 0)
    y, c = y[fin], c[fin]
    lo, hi = R.E2M1[R.e2m1_round(y * (1 - 2.0 ** -21))], R.E2M1[R.e2m1_round(y * (1 + 2.0 ** -21))]
    exact = R.E2M1[R.e2m1_round(y)]
    mag = np.abs(c)
    assert (mag == exact).all() if fmt == "mxfp4" else ((mag >= lo) & (mag <= hi)).all()
    assert ((np.sign(c) == np.sign(y)) | (c == 0)).all()
    # padding: zero codes past cols, zero scale bytes past the rows and blocks
    full = scales.reshape(scales.shape[0], scales.shape[1], 32, 4, 4).transpose(0, 3, 2, 1, 4)
    full = full.reshape(scales.shape[0] * 128, scales.shape[1] * 4)
    assert not full[rows:].any() and not full[:, nblk:].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 31), (33, 97), (127, 128), (129, 65),
                                       (300, 1000), (2, 8193)])
def test_quantize_and_back(B, fmt, dtype, rows, cols):
    import torch
    x = _x(rows, cols, rows + cols, dtype)
    g = _g(fmt)
    codes, scales = B.fp4_quantize(x, fmt, tensor_scale=g)
    _check_quantized(x.double().cpu().numpy(), codes.cpu().numpy(), scales.cpu().numpy(), fmt, g)
    want = R.values(codes.cpu().numpy(), scales.cpu().numpy(), fmt)[:, :cols]
    if g is not None:
        want = want * float(g)
    # element * scale * g is one rounding to fp32, then one to the output type
    want = torch.from_numpy(want.astype(np.float32))
    for o in ("f32", "f16", "bf16"):
        got = B.fp4_dequantize(codes, scales, cols, fmt, tensor_scale=g, dtype=_dt(o))
        assert torch.equal(got.cpu().float(), want.to(_dt(o)).float())


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_extremes(B, fmt):
    """Zero blocks, subnormal and huge values, ties, infinities and NaN."""
    import torch
    x = np.zeros((9, 64), np.float32)
    x[1, :] = 2.0 ** -149
    x[2, :8] = [3.4e38, -3.4e38, 1, -1, 0.5, 2.0 ** 126, 0, -0.0]
    # exactly on the midpoints for a block scale of 1
    x[3, :16] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 4]
    x[4, 5] = np.inf
    x[5, 40] = np.nan
    x[6, :] = np.linspace(-1, 1, 64)
    x[7, 63] = 2.0 ** -126
    x[8, 0] = -np.inf
    t = torch.from_numpy(x).cuda()
    codes, scales = B.fp4_quantize(t, fmt)
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    fin = [0, 2, 3, 6, 7] if fmt == "nvfp4" else [0, 1, 2, 3, 6, 7]
    _check = R.block_scales(x.astype(np.float64), fmt)
    assert np.array_equal(R.untile(s, 9, 64 // R.BLOCK[fmt])[fin], _check[fin])
    v = B.fp4_dequantize(codes, scales, 64, fmt).cpu().numpy()
    blk = R.BLOCK[fmt]
    nan = np.isnan(v.reshape(9, -1, blk))
    want = np.zeros_like(nan)
    want[4, 5 // blk] = want[5, 40 // blk] = want[8, 0] = True
    assert np.array_equal(nan, want)  # such a block reads back as NaN, its neighbours do not
    assert not v[0].any()
    if fmt == "mxfp4":
        assert list(v[3, 1:8]) == [0, 1, 1, 2, 2, 4, 4]
        assert list(v[3, 8:15]) == [0, -1, -1, -2, -2, -4, -4]


def test_quantize_strided_rows_and_given_outputs(B):
    import torch
    x = _x(70, 300, 5, "bf16")
    ref = B.fp4_quantize(x[:, 7:200].contiguous())
    got = B.fp4_quantize(x[:, 7:200])  # neither the base nor the rows on 16 bytes
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    rep = B.fp4_quantize(x[3:4].expand(40, 300))  # a repeated row
    one = B.fp4_quantize(x[3:4])
    assert torch.equal(rep[0], one[0].expand_as(rep[0]))
    out = [torch.full_like(t, 255) for t in ref]
    B.fp4_quantize(x[:, 7:200], codes=out[0], scales=out[1])
    assert all(torch.equal(a, b) for a, b in zip(ref, out))


def _bound(va, vb, alpha, cols):
    """Products of two elements and their scales are exact; adding cols of them
    in fp32, in whatever grouping, errs by at most cols / 16 + 4 units of 2^-23
    of the sum of magnitudes."""
    return (cols / 16 + 4) * 2.0 ** -23 * abs(alpha) * (np.abs(va) @ np.abs(vb).T)


def _operands(B, fmt, m, n, cols, seed):
    a, b = _x(m, cols, seed, "f32"), _x(n, cols, seed + 1, "f32")
    ga, gb = _g(fmt, 0.013), _g(fmt, 0.021)
    qa = B.fp4_quantize(a, fmt, tensor_scale=ga)
    qb = B.fp4_quantize(b, fmt, tensor_scale=gb)
    va, vb = (R.values(q[0].cpu().numpy(), q[1].cpu().numpy(), fmt) for q in (qa, qb))
    return qa, qb, ga, gb, va, vb


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,cols", [
    (1, 1, 1), (1, 128, 32), (2, 129, 96), (16, 1000, 64), (17, 257, 128), (33, 300, 300),
    (64, 128, 256), (65, 4099, 96), (128, 128, 512), (129, 1, 1000), (300, 515, 777),
    (1, 4096, 4096), (5, 333, 8200), (37, 2048, 2304), (130, 640, 4097), (513, 1283, 96),
    (100, 20000, 64), (100, 40000, 700), (1100, 2100, 1000), (130, 20000, 300), (300, 20000, 96),
    (1500, 20001, 160), (2500, 2500, 520), (257, 9999, 2050)])
def test_product(B, fmt, m, n, cols):
    """One row to many, ragged tiles and K, one and several K slices, few and
    many tiles per CTA."""
    import torch
    qa, qb, ga, gb, va, vb = _operands(B, fmt, m, n, cols, m + n + cols)
    alpha = 1.0 if ga is None else float(ga) * float(gb)
    want = alpha * (va @ vb.T)
    tol = _bound(va, vb, alpha, cols)
    got = B.fp4_product(*qa, *qb, fmt, a_tensor_scale=ga, b_tensor_scale=gb)
    assert got.dtype == torch.float32 and got.shape == (m, n)
    B.device_check()
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
    for o, u in (("bf16", 2.0 ** -8), ("f16", 2.0 ** -11)):
        h = B.fp4_product(*qa, *qb, fmt, a_tensor_scale=ga, b_tensor_scale=gb, dtype=_dt(o))
        assert torch.equal(h, got.to(_dt(o)))  # the same sums, rounded once
    again = B.fp4_product(*qa, *qb, fmt, a_tensor_scale=ga, b_tensor_scale=gb)
    assert torch.equal(got, again)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,cols", [(1, 300, 4096), (1, 32000, 100), (9, 515, 700),
                                      (40, 1000, 1111), (200, 640, 2048)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_linear_is_quantize_then_product(B, fmt, m, n, cols, dtype):
    import torch
    x = _x(m, cols, m, dtype)
    gx, gw = _g(fmt, 0.05), _g(fmt, 0.03)
    qw = B.fp4_quantize(_x(n, cols, n, "f32"), fmt, tensor_scale=gw)
    got = B.fp4_linear(x, *qw, fmt, x_tensor_scale=gx, w_tensor_scale=gw)
    qx = B.fp4_quantize(x, fmt, tensor_scale=gx)
    want = B.fp4_product(*qx, *qw, fmt, a_tensor_scale=gx, b_tensor_scale=gw, dtype=x.dtype)
    B.device_check()
    assert got.dtype == x.dtype
    vx = R.values(qx[0].cpu().numpy(), qx[1].cpu().numpy(), fmt)
    vw = R.values(qw[0].cpu().numpy(), qw[1].cpu().numpy(), fmt)
    alpha = 1.0 if gx is None else float(gx) * float(gw)
    unit = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    ref = alpha * (vx @ vw.T)
    tol = _bound(vx, vw, alpha, cols)
    # one rounding of each of the two to the output type besides; binary16's
    # least step is 2^-24
    lim = 2 * tol + unit * np.abs(ref) * 2 + (2.0 ** -24 if dtype == "f16" else 0)
    top = torch.finfo(x.dtype).max
    for y in (got, want):
        y = y.double().cpu().numpy()
        fin = np.isfinite(y)
        assert (np.abs(y - ref)[fin] <= lim[fin]).all()
        # infinite only where the result passes the type's largest, with its sign
        assert (np.abs(ref) + lim >= top)[~fin].all() and (np.sign(y) == np.sign(ref))[~fin].all()


def test_product_keeps_rows_apart(B):
    """A NaN block reaches its own row and column of the result only."""
    import torch
    a, b = _x(20, 256, 1, "f32"), _x(300, 256, 2, "f32")
    a[3, 100] = float("nan")
    b[299, 0] = float("inf")
    qa, qb = B.fp4_quantize(a), B.fp4_quantize(b)
    out = B.fp4_product(*qa, *qb)
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros((20, 300), bool)
    want[3, :] = want[:, 299] = True
    assert np.array_equal(nan, want)


def test_product_rows_of_a_larger_table(B):
    """128-row slices of packed rows are packed rows."""
    import torch
    qa, qb = B.fp4_quantize(_x(7, 200, 1, "f32")), B.fp4_quantize(_x(1000, 200, 2, "f32"))
    full = B.fp4_product(*qa, *qb)
    part = B.fp4_product(*qa, qb[0][256:640], qb[1][2:5])
    assert torch.equal(full[:, 256:640], part)


def test_empty(B):
    import torch
    e = torch.empty((0, 64), device="cuda")
    c, s = B.fp4_quantize(e)
    assert c.shape == (0, 32) and s.shape == (0, 1, 512)
    assert B.fp4_dequantize(c, s).shape == (0, 64)
    q = B.fp4_quantize(torch.ones((3, 64), device="cuda"))
    assert B.fp4_product(c, s, *q).shape == (0, 3)
    assert B.fp4_product(*q, c, s).shape == (3, 0)
    assert B.fp4_linear(e, *q).shape == (0, 3)


def test_on_another_stream(B):
    """Inputs made on the current stream, the call and its result on another."""
    import torch
    x = _x(64, 4096, 1, "bf16")
    qw = B.fp4_quantize(_x(1000, 4096, 2, "f32"))
    want = B.fp4_linear(x, *qw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = B.fp4_linear(x, *qw, stream=st)
    st.synchronize()
    assert torch.equal(got, want)


def test_output_past_32_bits(B):
    """More than 2^31 result elements: the last row is where it belongs."""
    import torch
    m, n = 33, 70_000_001
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 16 GB")
    a = torch.ones((m, 32), device="cuda")
    a[32] = 2.0
    qa = B.fp4_quantize(a)
    codes = torch.full((n, 16), 0x22, dtype=torch.uint8, device="cuda")  # every element 1
    scales = torch.zeros(B.fp4_shapes(n, 32)[1], dtype=torch.uint8, device="cuda")
    scales[:, :, :] = 127  # 2^0
    out = B.fp4_product(*qa, codes, scales, dtype=torch.bfloat16)
    B.device_check()
    assert bool((out[32, -1000:] == 64).all()) and bool((out[31, -1000:] == 32).all())
    assert bool((out[0, :1000] == 32).all())


@pytest.mark.parametrize("m,n,cols", [(301, 120_001, 64), (2100, 20_003, 96), (1111, 40_002, 2100)])
def test_large_results_at_odd_offsets(B, m, n, cols):
    """fp32 results past L2 whose rows start anywhere: the same values as the same
    product computed in column blocks, each result small and aligned."""
    import torch
    qa, qb = B.fp4_quantize(_x(m, cols, 1, "f32")), B.fp4_quantize(_x(n, cols, 2, "f32"))
    pad = torch.full((m * n + 3,), 7.0, device="cuda")
    out = pad[1:1 + m * n].view(m, n)  # 4 bytes past an aligned address
    B.fp4_product(*qa, *qb, out=out)
    B.device_check()
    assert float(pad[0]) == 7 and bool((pad[1 + m * n:] == 7).all())
    for c in range(0, n, 8192):
        e = min(n, c + 8192)
        part = B.fp4_product(*qa, qb[0][c:e], qb[1][c // 128:(e + 127) // 128])
        assert torch.equal(out[:, c:e], part)
