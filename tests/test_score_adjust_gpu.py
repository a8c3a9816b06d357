"""score_adjust against its definition in fp64."""

import numpy as np
import pytest

import scores_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from approximate_nearest_neighbour_gb300 import binding
    return binding


def _dt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _case(rows, cols, hist, nb, mask, seed):
    """Arguments as numpy arrays: skewed histories with entries out of range,
    lengths from none to all, repeated bias ids, a mask row that allows nothing."""
    r = np.random.default_rng(seed)
    a = {}
    if hist:
        a["history"] = (r.random((rows, hist)) ** 3 * cols).astype(np.int32)
        a["history"][r.random((rows, hist)) < 0.05] = -1
        a["history"][r.random((rows, hist)) < 0.02] = cols
        a["history_len"] = r.integers(0, hist + 1, rows).astype(np.int32)
        a["history_len"][0] = hist
        a["prompt_len"] = (a["history_len"] * r.random(rows)).astype(np.int32)
        a["repetition"] = (0.8 + r.random(rows)).astype(np.float32)
        a["presence"] = (r.random(rows) - 0.3).astype(np.float32)
        a["frequency"] = (r.random(rows) - 0.3).astype(np.float32)
    if nb:
        a["bias_ids"] = r.integers(-1, cols + 1, (rows, nb)).astype(np.int32)
        a["bias_ids"][:, -1] = a["bias_ids"][:, 0]
        a["bias_vals"] = r.standard_normal((rows, nb)).astype(np.float32) * 4
    a["temperature"] = (0.2 + r.random(rows)).astype(np.float32)
    if mask:
        m = r.integers(-2**31, 2**31, (1 if mask == "one" else rows, (cols + 31) // 32))
        a["mask"] = m.astype(np.int32)
        if mask == "rows" and rows > 1:
            a["mask"][1] = 0
    return a


def _cuda(a):
    import torch
    return {k: torch.from_numpy(v).cuda() for k, v in a.items()}


def _check(got, x, a, negate=False):
    """fp32 arithmetic of at most six roundings on values below the bound, and
    one rounding to the output type (binary16's least step is 2^-24)."""
    import torch
    want, mag = R.adjust(x.double().cpu().numpy(), negate=negate, **a)
    unit = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[got.dtype]
    g = got.double().cpu().numpy()
    fin = np.isfinite(want)
    assert np.array_equal(g[~fin], want[~fin], equal_nan=True)
    tol = 8 * 2.0 ** -24 * mag + unit * np.abs(np.where(fin, want, 0)) * 1.01
    tol += 2.0 ** -24 if got.dtype == torch.float16 else 2.0 ** -140
    assert (np.abs(g[fin] - want[fin]) <= tol[fin]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,hist,nb,mask,negate", [
    (1, 1, 1, 1, "one", False), (1, 32000, 200, 8, None, True), (3, 33, 70, 5, "rows", False),
    (5, 4096, 0, 0, "rows", False), (7, 4097, 1000, 0, None, False), (2, 70001, 5000, 300, "one", True),
    (64, 8191, 33, 17, "rows", False), (1, 200_000, 8192, 1, "rows", False),
    (300, 131, 9, 3, "one", False)])
def test_against_the_definition(B, dtype, rows, cols, hist, nb, mask, negate):
    import torch
    x = torch.from_numpy(np.random.default_rng(1).standard_normal((rows, cols)) * 4).to(_dt(dtype)).cuda()
    a = _case(rows, cols, hist, nb, mask, rows + cols)
    got = B.score_adjust(x, negate=negate, **_cuda(a))
    _check(got, x, a, negate)
    f32 = B.score_adjust(x, negate=negate, dtype=torch.float32, **_cuda(a))
    _check(f32, x, a, negate)
    again = B.score_adjust(x, negate=negate, dtype=torch.float32, **_cuda(a))
    assert torch.equal(f32.view(torch.int32), again.view(torch.int32))
    inplace = x.clone()
    B.score_adjust(inplace, negate=negate, out=inplace, **_cuda(a))
    assert torch.equal(inplace.view(torch.uint8), got.view(torch.uint8))


def test_single_arguments(B):
    """Each argument alone, and none."""
    import torch
    x = torch.randn(4, 501, device="cuda")
    a = _case(4, 501, 60, 7, "rows", 3)
    assert torch.equal(B.score_adjust(x), x)
    for keys in (["history", "repetition"], ["history", "presence"], ["history", "frequency"],
                 ["history", "history_len", "frequency"], ["history", "prompt_len", "presence"],
                 ["bias_ids", "bias_vals"], ["temperature"], ["mask"]):
        sub = {k: a[k] for k in keys}
        _check(B.score_adjust(x, **_cuda(sub)), x, sub)


def test_masked_places_hide_what_they_hold(B):
    """Infinities, NaN and the type's lowest value behind the mask, and beside it."""
    import torch
    x = torch.randn(3, 64, device="cuda", dtype=torch.float16)
    x[0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), -65504.0])
    mask = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    mask[0, 0] = -16  # columns 0 .. 3 are not allowed
    mask[2] = 0
    t = torch.full((3,), 0.5, device="cuda")
    out = B.score_adjust(x, mask=mask, temperature=t)
    assert bool((out[0, :4] == -float("inf")).all()) and bool(torch.isfinite(out[0, 4:]).all())
    assert bool((out[2] == -float("inf")).all())
    y = B.score_adjust(x, temperature=t)
    assert bool(torch.isnan(y[0, 0])) and float(y[0, 1]) == float("inf")
    assert float(y[0, 2]) == -float("inf") and float(y[0, 3]) == -float("inf")  # -131008 in binary16
    n = B.score_adjust(x, mask=mask, negate=True, dtype=torch.float32)
    v, i = B.kselect(n, 5)  # nothing masked is selected
    assert bool((i[0] >= 4).all()) and bool((v[2] == float("inf")).all())


def test_strided_and_repeated_rows(B):
    import torch
    base = torch.randn(6, 3000, device="cuda")
    x = base[:, 5:2006]
    a = _case(6, 2001, 100, 3, "rows", 9)
    c = _cuda(a)
    wide = torch.zeros((6, 300), dtype=torch.int32, device="cuda")
    wide[:, 17:117] = c["history"]
    c["history"] = wide[:, 17:117]
    want = B.score_adjust(x.contiguous(), **_cuda(a))
    assert torch.equal(B.score_adjust(x, **c), want)
    out = torch.full((6, 2500), 7.0, device="cuda")
    B.score_adjust(x, out=out[:, 3:2004], **c)
    assert torch.equal(out[:, 3:2004], want)
    assert bool((out[:, :3] == 7).all()) and bool((out[:, 2004:] == 7).all())
    one = B.score_adjust(x[2:3].expand(6, 2001), **c)
    assert torch.equal(one, B.score_adjust(x[2:3].expand(6, 2001).contiguous(), **c))


def test_empty(B):
    import torch
    assert B.score_adjust(torch.empty((0, 5), device="cuda")).shape == (0, 5)
    assert B.score_adjust(torch.empty((5, 0), device="cuda")).shape == (5, 0)
    x = torch.randn(2, 9, device="cuda")
    h = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    b = torch.empty((2, 0), device="cuda")
    assert torch.equal(B.score_adjust(x, history=h, bias_ids=h, bias_vals=b), x)


def test_rows_past_32_bits(B):
    """More than 2^31 scores in one call."""
    import torch
    rows, cols = 2200, 1_000_001
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-1, -1] = 3.0
    h = torch.full((rows, 1), cols - 1, dtype=torch.int32, device="cuda")
    p = torch.ones((rows,), device="cuda")
    B.score_adjust(x, history=h, presence=p, out=x)
    assert float(x[-1, -1]) == 2.0 and float(x[-2, -1]) == -1.0 and float(x[-1, -2]) == 0.0


def test_long_histories_and_bias_lists(B):
    """Past 32,767 tokens or 65,535 biases: counts of more than 15 bits, slots of more than 16."""
    import torch
    r = np.random.default_rng(8)
    x = torch.from_numpy(r.standard_normal((2, 5000)).astype(np.float32)).cuda()
    h = r.integers(0, 5000, (2, 70_000)).astype(np.int32)
    h[:, :50_000] = 3
    a = {"history": h, "prompt_len": np.array([49_000, 10], np.int32),
         "repetition": np.array([1.5, 0.7], np.float32),
         "presence": np.array([0.5, 0.25], np.float32),
         "frequency": np.array([1e-3, 2e-4], np.float32)}
    _check(B.score_adjust(x, **_cuda(a)), x, a)
    b = {"bias_ids": r.integers(-1, 5001, (2, 70_001)).astype(np.int32),
         "bias_vals": r.standard_normal((2, 70_001)).astype(np.float32)}
    _check(B.score_adjust(x, **_cuda(b)), x, b)
    both = {**a, **b, "mask": r.integers(-2**31, 2**31, (1, 157)).astype(np.int32)}
    _check(B.score_adjust(x, **_cuda(both)), x, both)
