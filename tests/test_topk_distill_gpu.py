"""topk_distill: loss and gradient against the definition in fp64 and differences."""

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


def _case(rows, cols, k, seed, repeated=False):
    """Scores, and lists with short tails, ids out of range and rows without any."""
    r = np.random.default_rng(seed)
    s = (r.standard_normal((rows, cols)) * 3).astype(np.float32)
    tv = np.sort(r.standard_normal((rows, k)).astype(np.float32) * 2, axis=1)
    if repeated:
        ti = r.integers(0, max(1, min(cols, k // 2 + 1)), (rows, k))
    else:
        ti = np.stack([r.permutation(cols)[:k] if cols >= k else
                       np.concatenate([r.permutation(cols), np.full(k - cols, -1)])
                       for _ in range(rows)])
    ti = ti.astype(np.int64)
    for row in range(0, rows, 3):
        n = int(r.integers(0, k + 1))
        tv[row, n:], ti[row, n:] = np.inf, -1  # as a search pads
    if rows > 4:
        ti[4, 0] = cols  # not a column
    g = r.standard_normal(rows).astype(np.float32)
    g[rows // 2] = 0 if rows > 2 else g[rows // 2]
    return s, tv, ti, g


def _run(B, s, tv, ti, g, tau, negated=True):
    import torch
    tvd, tid, gd = (torch.from_numpy(v).cuda() for v in (tv, ti, g))
    loss, stats = B.topk_distill_forward(s, tvd, tid, tau, negated=negated)
    grad = B.topk_distill_backward(s, tvd, tid, stats, gd, tau, negated=negated)
    loss2, grad2 = B.topk_distill(s, tvd, tid, gd, tau, negated=negated)
    return loss, stats, grad, loss2, grad2


def _check(out, s, tv, ti, g, tau, negated=True):
    """fp32 sums of up to cols / 256 + 64 terms in a row (chains per thread and
    the joins between them), exponentials of 2 ulp with an argument error of
    2^-22 of the distance from the maximum; one rounding to the output type."""
    import torch
    loss, stats, grad, loss2, grad2 = out
    s64 = s.double().cpu().numpy()
    wl, m, z, wg, dense = R.distill(s64, tv, ti, tau, negated, g)
    cols = s64.shape[1]
    e = (cols / 256 + 64) * 2.0 ** -24
    dist = np.abs(np.where(np.isfinite(s64), s64, 0) - np.where(np.isfinite(m), m, 0)[:, None]) / tau
    assert np.array_equal(stats[:, 0].double().cpu().numpy(), m)
    assert (np.abs(stats[:, 1].double().cpu().numpy() - z) <= (e + 2.0 ** -20) * z).all()
    # a loss is a sum of k products p (log p - log q): each log errs by e plus
    # 2^-22 of its size
    with np.errstate(over="ignore"):
        wl = np.where(np.isinf(wl.astype(np.float32)), np.inf, wl)  # past fp32's largest
    fin = np.isfinite(wl)
    tmax = np.abs(np.where(np.isfinite(tv), tv, 0)).max(1) * 2 / tau
    size = (tmax + dist.max(1) + np.log(cols) + 10) * (4 * 2.0 ** -22 + tv.shape[1] * 2.0 ** -24) + 2 * e
    for l in (loss, loss2):
        got = l.double().cpu().numpy()
        assert np.array_equal(got[~fin], wl[~fin], equal_nan=True)
        assert (np.abs(got[fin] - wl[fin]) <= tau * tau * size[fin]).all()
    assert torch.equal(loss, loss2)
    unit = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[grad.dtype]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(z[:, None] > 0, np.exp(-dist) / z[:, None], 0) * np.isfinite(s64)
    gw = np.abs(g[:, None]) * tau
    tol = gw * (q * (e + 2.0 ** -20 + dist * 2.0 ** -22) +
                dense * (tv.shape[1] * 2.0 ** -24 + 2.0 ** -20 + tmax[:, None] * 2.0 ** -22))
    tol = tol + unit * 1.01 * np.abs(wg) + (2.0 ** -25 if grad.dtype == torch.float16 else 2.0 ** -126)
    for x in (grad, grad2):
        assert x.dtype == s.dtype
        assert (np.abs(x.double().cpu().numpy() - wg) <= tol).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,k,tau", [
    (1, 1, 1, 1.0), (5, 7, 7, 2.0), (3, 5, 20, 1.0), (37, 32001, 10, 1.0), (8, 1000, 100, 0.25),
    (6, 4097, 2048, 4.0), (2, 200_003, 1000, 2.0), (300, 129, 3, 1.0), (9, 65536, 33, 1.0),
    (3, 131072, 64, 1.0), (2, 400_000, 20, 1.0), (2, 1_000_003, 50, 2.0)])
def test_against_the_definition(B, dtype, rows, cols, k, tau):
    import torch
    s, tv, ti, g = _case(rows, cols, k, rows + cols)
    t = torch.from_numpy(s).to(_dt(dtype)).cuda()
    out = _run(B, t, tv, ti, g, tau)
    _check(out, t, tv, ti, g, tau)
    again = _run(B, t, tv, ti, g, tau)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("rows,cols,k", [(7, 50, 9), (5, 3001, 300), (3, 40, 2048)])
def test_repeated_ids_add_up(B, rows, cols, k):
    import torch
    s, tv, ti, g = _case(rows, cols, k, 11, repeated=True)
    t = torch.from_numpy(s).cuda()
    _check(_run(B, t, tv, ti, g, 1.5), t, tv, ti, g, 1.5)


@pytest.mark.parametrize("negated", [False, True])
def test_sign_of_the_teacher(B, negated):
    import torch
    s, tv, ti, g = _case(6, 300, 17, 2)
    if not negated:
        tv = np.where(ti < 0, -np.inf, tv).astype(np.float32)
    t = torch.from_numpy(s).cuda()
    _check(_run(B, t, tv, ti, g, 1.0, negated), t, tv, ti, g, 1.0, negated)


def test_gradient_by_differences(B):
    """Central differences of the fp64 loss at the same scores; the reference's
    truncation error is h^2 times a bounded third derivative."""
    import torch
    s, tv, ti, g = _case(4, 23, 5, 7)
    g[:] = 1.0
    grad = B.topk_distill(torch.from_numpy(s).cuda(), *(torch.from_numpy(v).cuda() for v in (tv, ti, g)),
                          2.0, negated=True)[1].double().cpu().numpy()
    h = 1e-4
    for j in range(23):
        up, dn = s.astype(np.float64), s.astype(np.float64)
        up[:, j] += h
        dn[:, j] -= h
        d = (R.distill(up, tv, ti, 2.0, True)[0] - R.distill(dn, tv, ti, 2.0, True)[0]) / (2 * h)
        assert (np.abs(d - grad[:, j]) <= 2.0 ** -18 + 10 * h * h).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masked_scores(B, dtype):
    """-inf and the type's lowest value as masks, a listed masked column (its
    loss is infinite, its gradient is not), and rows with nothing left."""
    import torch
    s, tv, ti, g = _case(8, 600, 9, 3)
    g[:] = 1.0
    t = torch.from_numpy(s).to(_dt(dtype)).cuda()
    low = torch.finfo(t.dtype).min
    tv[[1, 2, 5, 7]] = np.linspace(0, 2, 9, dtype=np.float32)
    for r in (1, 2, 5, 7):
        ti[r] = np.arange(9) * 60 + r
    t[1, ::2] = -float("inf")
    t[1, ti[1]] = 1.0
    t[2, ti[2, 3]] = -float("inf")
    t[5] = -float("inf")
    t[7] = low
    t[6, ::3] = low
    for tau in (0.5, 2.0):
        _check(_run(B, t, tv, ti, g, tau), t, tv, ti, g, tau)


def test_nan_stays_in_its_row(B):
    import torch
    s, tv, ti, g = _case(5, 700, 6, 4)
    g[:] = 1.0
    g[3] = 0.0
    tv[:] = np.linspace(0, 1, 6, dtype=np.float32)
    ti[:] = np.arange(6) * 7
    t = torch.from_numpy(s).cuda()
    t[1, 500] = float("nan")
    t[3, 500] = float("nan")
    loss, stats, grad, loss2, grad2 = _run(B, t, tv, ti, g, 1.0)
    assert torch.isnan(loss).tolist() == [False, True, False, True, False]
    for x in (grad, grad2):
        assert bool(torch.isnan(x[1]).all()) and bool((x[3] == 0).all())  # a row that does not count
        assert bool(torch.isfinite(x[[0, 2, 4]]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,k", [(5, 1003, 20), (3, 70_001, 300)])
def test_in_place_and_strided(B, dtype, rows, cols, k):
    import torch
    s, tv, ti, g = _case(rows, cols, k, 6)
    base = torch.zeros((rows, cols + 37), dtype=_dt(dtype), device="cuda")
    base[:, 5:5 + cols] = torch.from_numpy(s).to(_dt(dtype)).cuda()
    x = base[:, 5:5 + cols]
    d = [torch.from_numpy(v).cuda() for v in (tv, ti, g)]
    loss, grad = B.topk_distill(x.contiguous(), *d, 2.0, negated=True)
    wide = torch.full((rows, cols + 9), 3.0, dtype=_dt(dtype), device="cuda")
    l2, _ = B.topk_distill(x, *d, 2.0, negated=True, grad=wide[:, 2:2 + cols])
    assert torch.equal(loss, l2) and torch.equal(wide[:, 2:2 + cols], grad)
    assert bool((wide[:, :2] == 3).all()) and bool((wide[:, 2 + cols:] == 3).all())
    _, stats = B.topk_distill_forward(x, *d[:2], 2.0, negated=True)
    y = x.contiguous()
    B.topk_distill_backward(y, *d[:2], stats, d[2], 2.0, negated=True, grad=y)
    assert torch.equal(y, B.topk_distill_backward(x, *d[:2], stats, d[2], 2.0, negated=True))
    B.topk_distill(x, *d, 2.0, negated=True, grad=x)
    assert torch.equal(x, grad) and bool((base[:, :5] == 0).all()) and bool((base[:, 5 + cols:] == 0).all())


def test_one_row_repeated(B):
    import torch
    s, tv, ti, g = _case(6, 900, 8, 1)
    x = torch.from_numpy(s).cuda()[2:3].expand(6, 900)
    d = [torch.from_numpy(v).cuda() for v in (tv, ti, g)]
    a, b = B.topk_distill(x, *d, negated=True), B.topk_distill(x.contiguous(), *d, negated=True)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_empty(B):
    import torch
    s = torch.empty((0, 10), device="cuda")
    tv, ti = torch.empty((0, 3), device="cuda"), torch.empty((0, 3), dtype=torch.int64, device="cuda")
    loss, grad = B.topk_distill(s, tv, ti, torch.empty((0,), device="cuda"))
    assert loss.shape == (0,) and grad.shape == (0, 10)
    loss, stats = B.topk_distill_forward(s, tv, ti)
    assert loss.shape == (0,) and stats.shape == (0, 2)


def test_a_search_as_the_teacher(B):
    """flat_knn's distances and ids as the list, its short tail included."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(1)
    db = torch.randn((12, 64), device="cuda", generator=gen)
    q = torch.randn((5, 64), device="cuda", generator=gen)
    dist, ids = B.flat_knn(db, q, 20)  # more than there are: (+inf, -1)
    s = -torch.cdist(q, db + 0.1)
    g = torch.ones(5, device="cuda")
    tv, ti = dist.cpu().numpy(), ids.cpu().numpy()
    out = _run(B, s, tv, ti, g.cpu().numpy(), 4.0)
    _check(out, s, tv, ti, g.cpu().numpy(), 4.0)


def test_more_rows_than_one_grid_dimension(B):
    """70,000 rows, the same 7,000 ten times."""
    import torch
    s, tv, ti, g = _case(7000, 40, 3, 5)
    d = [torch.from_numpy(v).cuda() for v in (s, tv, ti, g)]
    few = B.topk_distill(*d, 2.0, negated=True)
    d10 = [t.repeat(10, *([1] * (t.dim() - 1))) for t in d]
    many = B.topk_distill(*d10, 2.0, negated=True)
    loss, stats = B.topk_distill_forward(*d10[:3], 2.0, negated=True)
    grad = B.topk_distill_backward(*d10[:3], stats, d10[3], 2.0, negated=True)
    for t in range(10):
        at = slice(7000 * t, 7000 * (t + 1))
        assert torch.equal(many[0][at], few[0]) and torch.equal(many[1][at], few[1])
        assert torch.equal(loss[at], few[0]) and torch.equal(grad[at], few[1])
