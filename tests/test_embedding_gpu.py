"""embedding_lookup and embedding_gradient against their definitions."""

import numpy as np
import pytest

import decode_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from approximate_nearest_neighbour_gb300 import binding
    return binding


def _dt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _ids(tokens, rows, seed, wide=False):
    """Few tokens are frequent; some ids lie outside the table."""
    import torch
    r = np.random.default_rng(seed)
    i = (r.random(tokens) ** 4 * rows).astype(np.int64)
    i[r.random(tokens) < 0.1] = -1
    i[r.random(tokens) < 0.05] = rows
    if wide and tokens > 2:
        i[1] = 1 << 40
        i[2] = -(1 << 40) + rows // 2
    return torch.from_numpy(i if wide else i.astype(np.int32)).cuda()


def _rand(rows, cols, dtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((rows, cols), generator=g, device="cuda").to(_dt(dtype))


def _want_lookup(table, ids, scale, dtype):
    import torch
    i = ids.long()
    ok = (i >= 0) & (i < table.shape[0])
    x = table[torch.where(ok, i, 0)].float() * torch.tensor(scale, dtype=torch.float32, device="cuda")
    return torch.where(ok.unsqueeze(-1), x, 0.0).to(dtype)


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"),
                                       ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("tokens,rows,cols", [
    (1, 1, 1), (1, 100, 4096), (37, 1000, 4096), (5, 7, 3), (300, 50, 129), (64, 999, 101),
    (9000, 3001, 256), (5000, 2000, 1001), (3, 10, 70_001), (40_000, 500, 17)])
def test_lookup(B, dtype, out, tokens, rows, cols):
    """One product, rounded to fp32 and to the output: equal bits."""
    import torch
    t = _rand(rows, cols, dtype, tokens)
    for wide in (False, True):
        ids = _ids(tokens, rows, cols, wide)
        got = B.embedding_lookup(t, ids, 7.3, dtype=_dt(out))
        assert torch.equal(got, _want_lookup(t, ids, 7.3, _dt(out)))


def test_lookup_shapes_strides_and_streams(B):
    import torch
    big = _rand(60, 700, "bf16", 1)
    for off in (0, 1, 3, 8):
        t = big[:, off:off + 515]
        ids = _ids(35, 60, off)
        want = _want_lookup(t, ids, 1.0, torch.bfloat16)
        assert torch.equal(B.embedding_lookup(t, ids), want)
        room = torch.full((35, 600), 9.0, dtype=torch.bfloat16, device="cuda")
        B.embedding_lookup(t, ids, out=room[:, off:off + 515])
        assert torch.equal(room[:, off:off + 515], want)
        assert (room[:, :off] == 9).all() and (room[:, off + 515:] == 9).all()
    ids = _ids(24, 60, 5).view(2, 3, 4)
    got = B.embedding_lookup(big, ids, 0.5, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(got.view(24, 700), _want_lookup(big, ids.view(-1), 0.5, torch.bfloat16))
    one = big[:1].expand(60, 700)
    assert torch.equal(B.embedding_lookup(one, ids.view(-1)),
                       _want_lookup(one, ids.view(-1), 1.0, torch.bfloat16))
    assert B.embedding_lookup(big, ids[:0]).shape == (0, 3, 4, 700)
    none = torch.zeros((0, 8), device="cuda")
    assert torch.equal(B.embedding_lookup(none, ids.view(-1)), torch.zeros((24, 8), device="cuda"))


def _check_gradient(got, grad, ids, rows, scale, padding=-1, old=None):
    """fp32 sums of n terms, at most n - 1 additions in a row (rounded by half a step
    each, of a magnitude no larger than the terms'), the product with scale, the
    addition to what was there, and the rounding of the result."""
    import torch
    w, mag, count = R.gradient(grad.double().cpu().numpy(), ids.cpu().numpy().reshape(-1), rows,
                               scale, padding)
    tol = (count[:, None] + 2) * 2.0 ** -24 * mag
    if old is not None:
        o = old.double().cpu().numpy()
        w = w + o
        tol = np.where(count[:, None] > 0, tol + 2.0 ** -24 * np.abs(w), 0)
    half = torch.finfo(got.dtype).eps / 2
    tiny = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}[got.dtype]
    tol = tol * (1 + half) + half * np.abs(w) * (count[:, None] > 0) + tiny
    assert (np.abs(got.double().cpu().numpy() - w) <= tol).all()


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"),
                                       ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("tokens,rows,cols", [
    (1, 1, 1), (1, 300, 64), (31, 100, 33), (32, 1, 40), (33, 2, 9), (500, 129, 77),
    (777, 3001, 128), (3000, 40, 515), (5000, 20_000, 24), (64, 130, 3001)])
def test_gradient(B, dtype, out, tokens, rows, cols):
    import torch
    g = _rand(tokens, cols, dtype, rows)
    for wide in (False, True):
        ids = _ids(tokens, rows, tokens, wide)
        got = B.embedding_gradient(g, ids, rows, 3.5, dtype=_dt(out))
        _check_gradient(got, g, ids, rows, 3.5)
        assert torch.equal(got, B.embedding_gradient(g, ids, rows, 3.5, dtype=_dt(out)))
        old = _rand(rows, cols, out, 3)
        acc = old.clone()
        B.embedding_gradient(g, ids, rows, 3.5, accumulate=True, out=acc)
        _check_gradient(acc, g, ids, rows, 3.5, old=old)


def test_gradient_of_many_tokens(B):
    """Longer slabs; one token in all positions; all tokens different; none at all."""
    import torch
    g = _rand(70_000, 40, "f32", 1)
    for ids in (torch.zeros(70_000, dtype=torch.int32, device="cuda"),
                torch.randperm(70_000, device="cuda"),
                torch.full((70_000,), -1, dtype=torch.int32, device="cuda"),
                _ids(70_000, 70_000, 4)):
        _check_gradient(B.embedding_gradient(g, ids, 70_000), g, ids, 70_000, 1.0)


def test_gradient_of_many_frequent_tokens(B):
    """Hundreds of tokens of one class, each with more positions than are sorted by rank,
    with fewer, and with more than one block's list holds."""
    import torch
    g = _rand(60_000, 12, "f32", 3)
    r = np.random.default_rng(5)
    for step in (128, 1):
        for kinds in (300, 9):
            ids = torch.from_numpy((r.integers(0, kinds, 60_000) * step).astype(np.int32)).cuda()
            _check_gradient(B.embedding_gradient(g, ids, kinds * step), g, ids, kinds * step, 1.0)


def test_gradient_of_a_large_table(B):
    """More tokens per class than fit one block's counters at 128 classes."""
    import torch
    rows = (1 << 21) + 12_345
    g = _rand(3000, 4, "f32", 2)
    ids = _ids(3000, rows, 6)
    got = B.embedding_gradient(g, ids, rows)
    i = ids.long()
    ok = (i >= 0) & (i < rows)
    want = torch.zeros((rows, 4), dtype=torch.float64, device="cuda")
    want.index_put_((i[ok],), g[ok].double(), accumulate=True)
    mag = torch.zeros_like(want)
    mag.index_put_((i[ok],), g[ok].double().abs(), accumulate=True)
    assert bool(((got - want).abs() <= 300 * 2.0 ** -24 * mag).all())


def test_gradient_padding_strides_and_repeats(B):
    import torch
    big = _rand(200, 140, "bf16", 7)
    ids = _ids(200, 30, 8)
    for off in (0, 1, 5, 8):
        g = big[:, off:off + 101]
        room = torch.full((30, 120), 5.0, dtype=torch.bfloat16, device="cuda")
        B.embedding_gradient(g, ids, 30, 2.0, padding=0, out=room[:, 3:104])
        _check_gradient(room[:, 3:104].contiguous(), g, ids, 30, 2.0, padding=0)
        assert (room[:, :3] == 5).all() and (room[:, 104:] == 5).all()
        assert (room[0, 3:104] == 0).all()
    g = big[:1].expand(200, 140)  # the gradient of a broadcast output
    _check_gradient(B.embedding_gradient(g, ids, 30, dtype=torch.float32), g, ids, 30, 1.0)
    got = B.embedding_gradient(big, ids.view(10, 20), 30, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(got, B.embedding_gradient(big, ids, 30))
    e = B.embedding_gradient(big[:0], ids[:0], 30)
    assert e.shape == (30, 140) and (e == 0).all()
    assert B.embedding_gradient(big, ids, 0).shape == (0, 140)


def test_gradient_by_differences(B):
    """The lookup is linear in the table: a change of one entry by h changes
    <grad, lookup> by h times the gradient's entry."""
    import torch
    table = _rand(13, 6, "f32", 1).double()
    ids = _ids(50, 13, 2)
    g = _rand(50, 6, "f32", 3)
    d = B.embedding_gradient(g, ids, 13, 2.0).double()
    for v in range(13):
        for c in range(6):
            h = 0.5
            t2 = table.clone()
            t2[v, c] += h
            a, b = ((_want_lookup64(t, ids, 2.0) * g.double()).sum() for t in (t2, table))
            assert abs(float((a - b) / h - d[v, c])) <= 50 * 2.0 ** -24 * float(g.abs().sum())


def _want_lookup64(table, ids, scale):
    import torch
    i = ids.long()
    ok = (i >= 0) & (i < table.shape[0])
    return torch.where(ok.unsqueeze(-1), table[torch.where(ok, i, 0)] * scale, 0.0)


def test_captured_with_an_eager_one(B):
    """Two captured gradients, replayed in turn with new ids beside eager calls."""
    import torch
    g = _rand(600, 64, "bf16", 4)
    ids = [_ids(600, 200, i) for i in range(2)]
    B.embedding_gradient(g, ids[0], 200)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(B.embedding_gradient(g, ids[i], 200))
        graphs.append(graph)
    for round_ in range(3):
        for i in range(2):
            ids[i].copy_(_ids(600, 200, 10 + round_ * 2 + i))
            graphs[i].replay()
        eager = [B.embedding_gradient(g, v, 200) for v in ids]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))


@pytest.mark.parametrize("tokens", [200, 9000, 20_000])
@pytest.mark.parametrize("wide", [False, True])
def test_ids_at_any_offset(B, tokens, wide):
    """Ids that start off the 16-byte boundaries."""
    import torch
    g = _rand(tokens, 24, "f32", 1)
    ids = _ids(tokens, 300, 2, wide)
    want = B.embedding_gradient(g, ids, 300)
    table = _rand(300, 24, "f32", 3)
    rows = B.embedding_lookup(table, ids)
    for off in (1, 2, 3):
        room = torch.zeros(tokens + off, dtype=ids.dtype, device="cuda")
        room[off:] = ids
        assert torch.equal(B.embedding_gradient(g, room[off:], 300), want)
        assert torch.equal(B.embedding_lookup(table, room[off:]), rows)


def test_one_id(B):
    import torch
    table = _rand(9, 33, "f16", 1)
    i = torch.tensor(4, device="cuda")
    assert torch.equal(B.embedding_lookup(table, i), table[4])
    assert (B.embedding_lookup(table, i + 5) == 0).all()
