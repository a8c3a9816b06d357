"""beam_select and beam_reorder against their definitions."""

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


def _select(B, scores, totals, k, finished=None, end_id=0):
    import torch
    t = torch.from_numpy(totals).cuda()
    f = None if finished is None else torch.from_numpy(finished).cuda()
    got = B.beam_select(scores, t, k, finished=f, end_id=end_id)
    R.check_selection(got, scores.double().cpu().numpy(), totals, k, finished, end_id)
    again = B.beam_select(scores, t, k, finished=f, end_id=end_id)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    return got


def _scores(rows, cols, dtype, seed):
    import torch
    r = np.random.default_rng(seed)
    return torch.from_numpy((r.standard_normal((rows, cols)) * 3).astype(np.float32)).to(
        _dt(dtype)).cuda()


def _totals(groups, beams, seed):
    r = np.random.default_rng(seed + 1)
    t = -np.abs(r.standard_normal((groups, beams)) * 3).astype(np.float32)
    t[0, 1:] = -np.inf  # a group at its first token
    return t


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("groups,beams,cols,k", [
    (1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 7, 20), (1, 4, 32000, 8), (5, 5, 32001, 10),
    (3, 2, 129, 128), (2, 64, 300, 128), (1, 2, 200_003, 16), (70, 1, 1000, 3), (9, 3, 4099, 33),
    (400, 2, 257, 2), (4, 8, 70_000, 100)])
def test_against_the_definition(B, dtype, groups, beams, cols, k):
    s = _scores(groups * beams, cols, dtype, cols + k)
    _select(B, s, _totals(groups, beams, cols), k)


def test_rows_of_millions(B):
    """Batches of several loads per kept maximum."""
    _select(B, _scores(2, 3_000_001, "f32", 4), np.zeros((2, 1), np.float32), 50)
    _select(B, _scores(1, 5_000_000, "bf16", 5), np.zeros((1, 1), np.float32), 128)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [50, 5000, 131_072])
def test_equal_scores(B, dtype, cols):
    """Rows of one value throughout, of two, and of few: the lower columns come first."""
    import torch
    s = torch.zeros((6, cols), device="cuda")
    s[1] = 3.0
    s[2, ::7] = 1.0
    s[3, cols // 2:] = -1.0
    s[4] = torch.arange(cols, device="cuda") % 5
    s[5] = -(torch.arange(cols, device="cuda") // 3).float()
    s[0, ::2] = -0.0  # equal to +0
    for k in (1, 40, 128):
        _select(B, s.to(_dt(dtype)), np.array([[0, -1, -2, 0, -9, -1]], np.float32).T.copy(), k)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masks(B, dtype):
    """-inf and the type's lowest value as masks, rows of nothing else, NaN and +inf."""
    import torch
    low = torch.finfo(_dt(dtype)).min
    s = _scores(16, 3001, dtype, 8)
    m = torch.rand((16, 3001), device="cuda") < 0.9
    s[0:2] = torch.where(m[0:2], -float("inf"), s[0:2])
    s[2:4] = torch.where(m[2:4], low, s[2:4])
    s[4] = -float("inf")
    s[5] = low
    s[6] = -float("inf")
    s[6, 77] = 1.0            # one continuation
    s[7] = low
    s[7, [5, 2000]] = -float("inf")
    s[8, 100] = float("nan")
    s[9, 3000] = float("inf")
    s[10] = -float("inf")
    s[10, 9] = float("nan")
    s[11, 40] = torch.finfo(_dt(dtype)).max
    s[12] = low
    s[12, :5] = torch.finfo(_dt(dtype)).max
    for groups in (1, 4, 16):
        _select(B, s, np.zeros((groups, 16 // groups), np.float32) - 0.5, 20)


def test_dead_and_finished_beams(B):
    import torch
    s = _scores(24, 500, "bf16", 3)
    s[5] = float("nan")  # a finished beam's scores are not read
    t = _totals(6, 4, 9)
    t[1] = -np.inf        # nothing alive
    t[2, 0], t[2, 1], t[2, 2] = np.nan, np.inf, -np.inf
    f = np.zeros((6, 4), np.uint8)
    f[1] = 1
    f[:, 1] = 1
    f[3] = 7              # all finished
    got = _select(B, s, t, 9, f, 499)
    assert (got[1][1] == -1).all()
    assert int((got[1][3] >= 0).sum()) == 4 and (got[2][3, :4] == 499).all()
    b = B.beam_select(s, torch.from_numpy(t).cuda(), 9, finished=torch.from_numpy(f != 0).cuda(),
                      end_id=499)
    assert all(torch.equal(x, y) for x, y in zip(got, b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_repeated_rows(B, dtype):
    """Rows inside a wider matrix at any offset give the same bits; beams that share a
    row have equal totals, and the lower beam comes first."""
    import torch
    s = _scores(12, 4001, dtype, 6)
    t = _totals(3, 4, 2)
    want = _select(B, s, t, 13)
    wide = torch.zeros((12, 4100), dtype=s.dtype, device="cuda")
    for off in range(0, 9):
        wide[:, off:off + 4001] = s
        got = B.beam_select(wide[:, off:off + 4001], torch.from_numpy(t).cuda(), 13)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    one = s[:1].expand(8, 4001)
    got = _select(B, one, np.zeros((2, 4), np.float32), 10)
    assert got[1][0].tolist() == [0, 1, 2, 3, 0, 1, 2, 3, 0, 1] or dtype == "bf16"
    i = got[2][0].tolist()
    b = got[1][0].tolist()
    lists = got[0][0].tolist()
    assert all(lists[j] > lists[j + 1] or (b[j], i[j]) < (b[j + 1], i[j + 1]) for j in range(9))


def test_empty_and_streams(B):
    import torch
    e = B.beam_select(torch.zeros((0, 5), device="cuda"), torch.zeros((0, 3), device="cuda"), 4)
    assert [tuple(v.shape) for v in e] == [(0, 4)] * 3
    s = _scores(40, 20_000, "bf16", 11)
    t = torch.from_numpy(_totals(10, 4, 1)).cuda()
    want = B.beam_select(s, t, 8)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [B.beam_select(s, t, 8, stream=streams[i % 4]) for i in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in got for a, b in zip(o, want))


def test_captured_with_a_second_kernel(B):
    """More entries than one cluster ranks: two kernels and workspace in a graph."""
    import torch
    s = _scores(40, 9000, "bf16", 20)
    t = torch.from_numpy(_totals(2, 20, 1)).cuda()
    B.beam_select(s, t, 40)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = B.beam_select(s, t, 40)
    for i in range(3):
        s.copy_(_scores(40, 9000, "bf16", 30 + i))
        g.replay()
        want = B.beam_select(s, t, 40)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_captured(B):
    """Selection and in-place reordering captured; two graphs replayed in turn."""
    import torch
    s = [_scores(12, 9000, "f16", 20 + i) for i in range(2)]
    t = [torch.from_numpy(_totals(3, 4, i)).cuda() for i in range(2)]
    st = [torch.randn((12, 5, 64), device="cuda") for _ in range(2)]
    B.beam_select(s[0], t[0], 4)  # loaded before the capture
    B.beam_reorder(st[0].clone(), torch.zeros((3, 4), dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = B.beam_select(s[i], t[i], 4)
            B.beam_reorder(st[i], o[1])
        graphs.append(g)
        outs.append(o)
    for round_ in range(3):
        for i in (0, 1):
            s[i].copy_(_scores(12, 9000, "f16", 50 + 2 * round_ + i))
            before = st[i].clone()
            graphs[i].replay()
            torch.cuda.synchronize()
            want = B.beam_select(s[i], t[i], 4)
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want))
            rows = want[1].long() + torch.arange(3, device="cuda").unsqueeze(1) * 4
            assert torch.equal(st[i], before[rows.view(-1)])


# ---- reordering ------------------------------------------------------------------
def _want(state, out, beams, width, lengths, axis):
    """The definition, row by row."""
    w = out.clone()
    groups, n = beams.shape
    for g in range(groups):
        for j in range(n):
            b = int(beams[g, j])
            if not 0 <= b < width:
                continue
            src, dst = state[g * width + b], w[g * n + j]
            if lengths is None:
                dst.copy_(src)
            else:
                m = max(0, min(int(lengths[g]), state.shape[axis]))
                dst.narrow(axis - 1, 0, m).copy_(src.narrow(axis - 1, 0, m))
    return w


def _random(shape, dtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    if dtype.is_floating_point:
        return torch.randn(shape, generator=g, device="cuda").to(dtype)
    return torch.randint(-100, 100, shape, generator=g, device="cuda").to(dtype)


def _beams(groups, width, n, seed, invalid=True):
    import torch
    r = np.random.default_rng(seed)
    b = r.integers(-2 if invalid else 0, width + (2 if invalid else 0), (groups, n))
    return torch.from_numpy(b.astype(np.int32)).cuda()


@pytest.mark.parametrize("groups,width,n", [(1, 1, 1), (1, 4, 4), (3, 5, 5), (2, 64, 64),
                                            (4, 1, 6), (2, 6, 3), (7, 2, 2)])
@pytest.mark.parametrize("name", ["bfloat16", "float32", "int32", "uint8", "int64", "int16"])
def test_reorder(B, groups, width, n, name):
    import torch
    dt = getattr(torch, name)
    shapes = [(3, 40, 16), (37,), (2, 1000, 8), (1, 1, 1)]
    states = [_random((groups * width, *s), dt, i) for i, s in enumerate(shapes)]
    axes = [2, 1, 2, 3]
    beams = _beams(groups, width, n, 5)
    r = np.random.default_rng(3)
    some = torch.from_numpy(r.integers(-1, 1100, groups).astype(np.int32)).cuda()
    for lengths in (None, some):
        outs = [_random((groups * n, *s), dt, 10 + i) for i, s in enumerate(shapes)]
        want = [_want(t, o, beams, width, lengths, a) for t, o, a in zip(states, outs, axes)]
        keep = [t.clone() for t in states]
        got = B.beam_reorder(states, beams, lengths=lengths, axis=axes, out=outs)
        assert got is outs and all(torch.equal(a, b) for a, b in zip(outs, want))
        assert all(torch.equal(a, b) for a, b in zip(states, keep))
        if width == n:
            want = [_want(t, t, beams, width, lengths, a) for t, a in zip(states, axes)]
            mine = [t.clone() for t in states]
            assert B.beam_reorder(mine, beams, lengths=lengths, axis=axes) is mine
            assert all(torch.equal(a, b) for a, b in zip(mine, want))


def test_reorder_many_states_and_views(B):
    """More states than one launch takes; keys and values interleaved in one buffer;
    rows that are not dense; a source row that is repeated."""
    import torch
    beams = _beams(3, 4, 4, 8, invalid=False)
    states = [_random((12, 2, 50 + i, 8), torch.float16, i) for i in range(70)]
    lengths = torch.tensor([0, 17, 200], dtype=torch.int32, device="cuda")
    want = [_want(t, t, beams, 4, lengths, 2) for t in states]
    B.beam_reorder(states, beams, lengths=lengths, axis=2)
    assert all(torch.equal(a, b) for a, b in zip(states, want))
    both = _random((12, 2, 3, 40, 16), torch.bfloat16, 1)
    want = both.clone()
    for i in range(2):
        want[:, i] = _want(both[:, i], both[:, i], beams, 4, lengths, 2)
    B.beam_reorder([both[:, 0], both[:, 1]], beams, lengths=lengths, axis=2)
    assert torch.equal(both, want)
    wide = _random((12, 30), torch.int16, 2)
    part = wide[:, 3:20]
    want = wide.clone()
    want[:, 3:20] = _want(part, part, beams, 4, None, 1)
    B.beam_reorder(part, beams)
    assert torch.equal(wide, want)
    row = _random((1, 33), torch.float32, 3).expand(12, 33)
    out = torch.zeros((12, 33), device="cuda")
    B.beam_reorder(row, beams, out=out)
    assert torch.equal(out, row)


def test_reorder_far_offsets(B):
    """Rows whose offsets pass 32 bits."""
    import torch
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 12 GB")
    t = torch.zeros((4, 3, 1 << 29), dtype=torch.uint8, device="cuda")
    for i in range(4):
        t[i, 2, -100:] = i + 1
        t[i, 0, :100] = i + 11
    beams = torch.tensor([[3, 3, 0, 1]], dtype=torch.int32, device="cuda")
    n = torch.tensor([1 << 29], dtype=torch.int32, device="cuda")
    B.beam_reorder(t, beams, lengths=n, axis=2)
    assert t[:, 2, -100:].amax(1).tolist() == [4, 4, 1, 2]
    assert t[:, 0, :100].amin(1).tolist() == [14, 14, 11, 12] and int(t[:, 1].max()) == 0


def test_reorder_refusals_of_the_binding(B):
    import torch
    beams = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    t = torch.zeros((6, 4, 5), device="cuda")
    lengths = torch.ones((2,), dtype=torch.int32, device="cuda")
    bad = [lambda: B.beam_reorder(t[:4], beams),                       # in place, other width
           lambda: B.beam_reorder(t[:5], beams),                       # not whole groups
           lambda: B.beam_reorder([t, t], beams),                      # written twice
           lambda: B.beam_reorder(t, beams, out=torch.zeros((6, 4, 6), device="cuda")),
           lambda: B.beam_reorder([t], beams, out=[t.clone(), t.clone()]),
           lambda: B.beam_reorder(t, beams, lengths=lengths[:1]),
           lambda: B.beam_reorder(t, beams, lengths=lengths, axis=3),
           lambda: B.beam_reorder(t, beams, lengths=lengths, axis=0),
           lambda: B.beam_reorder(t.transpose(1, 2), beams, lengths=lengths, axis=1),
           lambda: B.beam_reorder(torch.zeros((6, 4, 5, 6), device="cuda").transpose(1, 3)[:, 1:],
                                  beams),
           lambda: B.beam_reorder(torch.zeros((1, 5), device="cuda").expand(6, 5), beams),
           lambda: B.beam_reorder(t, torch.zeros((2, 65), dtype=torch.int32, device="cuda"),
                                  out=torch.zeros((130, 4, 5), device="cuda")),
           lambda: B.beam_reorder(t.cpu(), beams)]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, B.IVFPQError)):
            call()
            pytest.fail(f"case {i} was taken")
    with pytest.raises(TypeError):
        B.beam_reorder(t, beams.long())


@pytest.mark.parametrize("beams", range(1, 18))
def test_every_number_of_beams(B, beams):
    """A cluster per group up to 16 beams with few continuations, and both ways of ranking."""
    for groups, cols, k in ((3, 20_000, 3), (2, 5000, 16), (40, 700, 2 * beams)):
        r = np.random.default_rng(beams)
        t = -np.abs(r.standard_normal((groups, beams)) * 2).astype(np.float32)
        t[0, beams // 2] = -np.inf
        f = (r.random((groups, beams)) < 0.2).astype(np.uint8)
        _select(B, _scores(groups * beams, cols, "bf16", beams + cols), t, min(k, 128), f, 5)


def test_the_two_ways_agree(B):
    """A selection of few continuations is the beginning of one of many: one cluster
    ranks the first, two kernels the second."""
    import torch
    for dtype in ("f32", "bf16"):
        s = _scores(24, 6001, dtype, 2)
        s[3] = s[2]  # equal rows: the lower beam comes first
        t = torch.zeros((6, 4), device="cuda")
        few, many = B.beam_select(s, t, 8), B.beam_select(s, t, 128)
        assert all(torch.equal(a, b[:, :8]) for a, b in zip(few, many))
