"""adapter_linear against its definition."""

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


def _case(tokens, cols, n, rank, adapters, dtype, out, seed, runs=False):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    r = np.random.default_rng(seed)
    ids = r.integers(-1, adapters + 1, tokens).astype(np.int32)
    if runs:
        ids = np.sort(ids)[::-1].copy()
    return dict(x=rn(tokens, cols).to(_dt(dtype)), a=(rn(adapters, rank, cols) * cols ** -0.5).to(_dt(dtype)),
                b=rn(adapters, n, rank).to(_dt(dtype)), ids=torch.from_numpy(ids).cuda(),
                scales=rn(adapters).abs() + 0.5, base=rn(tokens, n).to(_dt(out)))


def _check(got, x, a, b, ids, scales, base):
    """The first product: fp32 sums whose longest chain is cols / 64 instructions of 16
    terms (each may lose 2^-22 of the terms' magnitudes) and the joins; its cut into
    terms of the type: 2^-16 (2^-22 for fp32 outputs) of each element; the second
    product: at most 8 instructions for each of 3 terms, the same loss; the sum with
    base, and the rounding of the result."""
    import torch
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    w, second, first = R.adapter(f(x), f(a), f(b), ids.cpu().numpy(), f(scales), f(base))
    cols, wide = x.shape[1], got.dtype == torch.float32
    half = torch.finfo(got.dtype).eps / 2
    tol = first * (cols / 64 + 32) * 2.0 ** -22 + second * ((2.0 ** -22 if wide else 2.0 ** -16) + 26 * 2.0 ** -22)
    tol = tol * (1 + half) + (half + 2.0 ** -24) * np.abs(w) + (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -133)
    assert got.shape == w.shape
    assert (np.abs(f(got) - w) <= tol).all(), np.abs(f(got) - w).max()


@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"),
                                       ("bf16", "f32")])
@pytest.mark.parametrize("tokens,cols,n,rank,adapters", [
    (1, 1, 1, 1, 1), (1, 4096, 300, 16, 3), (3, 64, 40, 8, 2), (16, 512, 129, 4, 5),
    (17, 512, 129, 4, 5), (5, 77, 33, 3, 2), (40, 1001, 65, 24, 6), (77, 256, 512, 16, 64),
    (33, 96, 64, 64, 1), (70, 200, 250, 128, 3), (30, 136, 1000, 100, 2), (300, 128, 200, 32, 4),
    (520, 160, 320, 16, 3), (9, 40, 31, 17, 2), (300, 96, 200, 4, 2), (300, 96, 201, 100, 2),
    (100, 96, 72, 100, 2), (130, 64, 72, 128, 1), (64, 200, 136, 40, 2), (257, 72, 1030, 9, 3)])
def test_against_the_definition(B, dtype, out, tokens, cols, n, rank, adapters):
    import torch
    c = _case(tokens, cols, n, rank, adapters, dtype, out, tokens + cols + n)
    got = B.adapter_linear(**c)
    _check(got, **c)
    assert torch.equal(got, B.adapter_linear(**c))
    room = torch.full((tokens, n + 9), 3.0, dtype=_dt(out), device="cuda")
    room[:, 5:5 + n] = c["base"]
    view = room[:, 5:5 + n]
    d = dict(c, base=view, out=view)  # in place, inside wider rows
    assert B.adapter_linear(**d) is view
    assert torch.equal(view, got) and (room[:, :5] == 3).all() and (room[:, 5 + n:] == 3).all()
    d = dict(c, base=None, scales=None, dtype=_dt(out))
    _check(B.adapter_linear(**d), **{k: v for k, v in d.items() if k != "dtype"})


def test_tokens_do_not_depend_on_their_neighbours(B):
    """A token's row is the same whatever tile it falls into."""
    import torch
    c = _case(400, 320, 200, 16, 3, "bf16", "bf16", 5, runs=True)
    want = B.adapter_linear(**c)
    order = torch.randperm(400, device="cuda")
    d = dict(c, x=c["x"][order].contiguous(), ids=c["ids"][order].contiguous(),
             base=c["base"][order].contiguous())
    assert torch.equal(B.adapter_linear(**d), want[order])


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_strides_and_repeats(B, tokens):
    import torch
    c = _case(tokens, 264, 96, 16, 4, "bf16", "bf16", 9)
    want = B.adapter_linear(**c)
    wide = torch.zeros((tokens, 300), dtype=torch.bfloat16, device="cuda")
    for off in range(9):
        wide[:, off:off + 264] = c["x"]
        assert torch.equal(B.adapter_linear(**dict(c, x=wide[:, off:off + 264])), want)
    one = c["x"][:1].expand(tokens, 264)
    row = c["base"][:1].expand(tokens, 96)
    d = dict(c, x=one, base=row)
    _check(B.adapter_linear(**d), **d)


@pytest.mark.parametrize("tokens", [4, 50])
def test_no_adapters_and_none_used(B, tokens):
    import torch
    c = _case(tokens, 64, 48, 8, 2, "f16", "f16", 1)
    none = torch.full((tokens,), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(B.adapter_linear(**dict(c, ids=none)), c["base"])
    z = B.adapter_linear(**dict(c, ids=none, base=None))
    assert (z == 0).all() and z.dtype == torch.float16
    d = dict(c, a=c["a"][:0], b=c["b"][:0], scales=c["scales"][:0])
    assert torch.equal(B.adapter_linear(**d), c["base"])
    far = torch.full((tokens,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    assert torch.equal(B.adapter_linear(**dict(c, ids=far)), c["base"])
    e = dict(c, x=c["x"][:0], ids=c["ids"][:0], base=c["base"][:0])
    assert B.adapter_linear(**e).shape == (0, 48)


def test_small_and_large_values(B):
    """fp16 operands whose inner products lie outside fp16's range, and a row of zeros."""
    import torch
    c = _case(60, 128, 64, 16, 3, "f16", "f32", 2)
    for f, s in ((200.0, 1e-3), (2.0 ** -14, 1.0), (1.0, 1e6), (1.0, 1e-8)):
        d = dict(c, x=(c["x"].float() * f).half(), scales=c["scales"] * s)
        d["x"][3] = 0
        _check(B.adapter_linear(**d), **d)


def test_infinities_stay_in_their_rows(B):
    import torch
    c = _case(40, 64, 32, 8, 2, "bf16", "bf16", 3)
    want = B.adapter_linear(**c)
    c["x"][7, 5] = float("inf")
    c["x"][30, 0] = float("nan")
    got = B.adapter_linear(**c)
    for t in range(40):
        if t not in (7, 30):
            assert torch.equal(got[t], want[t])
    for t in (7, 30):
        if 0 <= int(c["ids"][t]) < 2:
            assert not torch.isfinite(got[t]).any()


def test_streams_and_captured(B):
    import torch
    cs = [_case(t, 256, 300, 16, 5, "bf16", "bf16", t) for t in (3, 50, 700)]
    want = [B.adapter_linear(**c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(10):
        got = [B.adapter_linear(**c, stream=s) for c, s in zip(cs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for c in cs[1:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(B.adapter_linear(**c))
        graphs.append(g)
    for _ in range(2):
        for c in cs[1:]:
            c["ids"].copy_(c["ids"].flip(0))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, o in zip(cs[1:], outs):
            assert torch.equal(o, B.adapter_linear(**c))


def test_operands_at_any_offset(B):
    """Adapters that start off the 16-byte boundaries give the same results, but where
    tiles of 128 tokens then take another product: there within its error."""
    import torch
    for tokens, rank in ((30, 16), (30, 24), (300, 16), (100, 64)):
        c = _case(tokens, 136, 72, rank, 2, "bf16", "f32", 4)
        want = B.adapter_linear(**c)
        for off in (1, 3, 8):
            d = dict(c)
            for name in ("a", "b"):
                flat = torch.zeros(c[name].numel() + off, dtype=torch.bfloat16, device="cuda")
                d[name] = flat[off:].view(c[name].shape)
                d[name].copy_(c[name])
            got = B.adapter_linear(**d)
            _check(got, **d)
            if tokens < 64:
                assert torch.equal(got, want)


def test_rows_of_one_value(B):
    """Every token the same: every result the same, whatever its place in a tile."""
    import torch
    for tokens in (1, 2, 15, 16, 17, 255, 256, 257, 384, 385):
        c = _case(tokens, 64, 40, 8, 1, "f16", "f32", 3)
        c["ids"].zero_()
        c["x"].copy_(c["x"][:1].expand(tokens, 64).clone())
        c["base"].copy_(c["base"][:1].expand(tokens, 40).clone())
        got = B.adapter_linear(**c)
        assert torch.equal(got, got[:1].expand(tokens, 40))
        _check(got, **c)


@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"),
                                       ("bf16", "f32")])
@pytest.mark.parametrize("rank", [24, 72])
def test_rows_at_any_offset(B, dtype, out, rank):
    """Base rows and output rows that start anywhere, each at its own offset, of full and
    of last units: the same results to the bit, and nothing beside them is written."""
    import torch
    for n in (1, 2, 3, 63, 64, 127, 128, 129, 255, 257, 386):
        c = _case(300, 64, n, rank, 2, dtype, out, n, runs=True)
        want = B.adapter_linear(**c)
        _check(want, **c)
        for i, o, wide in ((0, 1, 1), (1, 0, 1), (1, 1, 2), (2, 3, 2), (3, 2, 4), (7, 8, 8)):
            base = torch.full((300 * (n + wide) + i,), 7.0, dtype=_dt(out), device="cuda")
            base = base[i:].view(300, n + wide)[:, :n]
            base.copy_(c["base"])
            room = torch.full((1 + o + 300 * (n + wide),), 3.0, dtype=_dt(out), device="cuda")
            rows = room[1 + o:].view(300, n + wide)
            B.adapter_linear(**dict(c, base=base, out=rows[:, :n]))
            assert torch.equal(rows[:, :n], want), (n, i, o, wide)
            assert (room[:1 + o] == 3).all() and (rows[:, n:] == 3).all()
            B.adapter_linear(**dict(c, base=base, out=base))
            assert torch.equal(base, want), (n, i, o, wide)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rank", [8, 24, 128])
def test_odd_columns(B, dtype, rank):
    """Rows of x and of the adapters that start anywhere and end inside a vector: to the
    bit what the same rows with zeros behind them give."""
    import torch
    for cols in (1, 7, 63, 65, 71, 127, 129, 1001):
        c = _case(300, cols, 96, rank, 2, dtype, "f32", cols, runs=True)
        got = B.adapter_linear(**c)
        _check(got, **c)
        more = -cols % 8
        d = dict(c, **{k: torch.nn.functional.pad(c[k], (0, more)) for k in ("x", "a")})
        assert torch.equal(B.adapter_linear(**d), got), cols
        # what lies beside the rows, infinities even, is not looked at
        room = torch.full((300, cols + 9), float("inf"), dtype=_dt(dtype), device="cuda")
        for off in (1, 4, 9):
            room.fill_(float("inf"))
            room[:, off:off + cols] = c["x"]
            assert torch.equal(B.adapter_linear(**dict(c, x=room[:, off:off + cols])), got), cols
