"""Host-side refusals of the beam, embedding and adapter entry points."""

import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from approximate_nearest_neighbour_gb300 import binding, build
    build.build_library()
    return binding.lib()


def _bad(lib, calls):
    from approximate_nearest_neighbour_gb300 import binding as B
    for i, call in enumerate(calls):
        rc = call()
        assert rc == B.IVFPQ_ERR_INVALID_ARG, (i, rc)
        assert lib.ivfpq_last_error(), i


P = C.c_void_p(256)


def test_select_refusals(lib):
    def call(scores=P, dtype=0, groups=2, beams=3, cols=8, lds=8, totals=P, fin=None, end=0, k=4,
             ot=P, ob=P, oi=P):
        return lib.beam_select(scores, dtype, groups, beams, cols, lds, totals, fin, end, k, ot, ob,
                               oi, None)
    _bad(lib, [lambda: call(dtype=3), lambda: call(groups=-1), lambda: call(beams=0),
               lambda: call(beams=65), lambda: call(groups=1 << 31), lambda: call(groups=1 << 30),
               lambda: call(groups=1 << 62), lambda: call(cols=0), lambda: call(cols=(1 << 28) + 1),
               lambda: call(lds=7), lambda: call(k=0), lambda: call(k=129),
               lambda: call(scores=None), lambda: call(totals=None), lambda: call(ot=None),
               lambda: call(ob=None), lambda: call(oi=None), lambda: call(fin=P, end=8),
               lambda: call(fin=P, end=-1)])
    assert call(groups=0, scores=None) == 0


def test_reorder_refusals(lib):
    from approximate_nearest_neighbour_gb300 import binding as B

    def call(n=3, width=3, groups=2, count=1, beams=P, lengths=None, states=True, **kw):
        f = dict(src=256, dst=512, src_row=64, dst_row=64, outer=1, src_outer=0, dst_outer=0,
                 inner=64, unit=0)
        f.update(kw)
        a = (C.c_int64 * B._STATE)(*(v or 0 for v in f.values()))
        return lib.beam_reorder(a if states else None, count, beams, groups, width, n, lengths, None)
    _bad(lib, [lambda: call(n=0), lambda: call(n=65), lambda: call(width=0), lambda: call(width=65),
               lambda: call(groups=-1), lambda: call(groups=1 << 26), lambda: call(count=-1),
               lambda: call(beams=None), lambda: call(states=False), lambda: call(src=None),
               lambda: call(dst=None), lambda: call(src_row=-1), lambda: call(dst_row=-64),
               lambda: call(dst_row=63), lambda: call(outer=2, dst_outer=32), lambda: call(inner=-1),
               lambda: call(inner=1 << 40, dst_row=1 << 41), lambda: call(outer=1 << 31),
               lambda: call(unit=-1), lambda: call(dst=256, n=2),
               lambda: call(dst=256, src_row=128),
               lambda: call(dst=256, outer=2, src_outer=64, dst_outer=128, src_row=256, dst_row=256)])
    assert call(groups=0) == 0 and call(count=0) == 0 and call(outer=0) == 0 and call(inner=0) == 0


def test_embedding_refusals(lib):
    def look(table=P, dtype=0, rows=9, cols=8, ldt=8, ids=P, size=4, tokens=5, out=P, odt=0, ldo=8):
        return lib.embedding_lookup(table, dtype, rows, cols, ldt, ids, size, tokens, 1.0, out, odt,
                                    ldo, None)

    def grad(g=P, dtype=0, tokens=5, cols=8, ldg=8, ids=P, size=8, rows=9, acc=0, out=P, odt=0,
             ldo=8):
        return lib.embedding_gradient(g, dtype, tokens, cols, ldg, ids, size, rows, 1.0, -1, acc, out,
                                      odt, ldo, None)
    for f in (look, grad):
        _bad(lib, [lambda: f(dtype=3), lambda: f(odt=7), lambda: f(odt=1), lambda: f(dtype=1, odt=2),
                   lambda: f(rows=-1), lambda: f(rows=(1 << 24) + 1), lambda: f(cols=-1),
                   lambda: f(cols=(1 << 20) + 1), lambda: f(tokens=-1), lambda: f(tokens=1 << 30),
                   lambda: f(size=2), lambda: f(ids=None), lambda: f(out=None), lambda: f(ldo=7)])
    _bad(lib, [lambda: look(ldt=7), lambda: look(table=None), lambda: grad(ldg=7),
               lambda: grad(g=None)])
    assert look(tokens=0) == 0 and look(cols=0) == 0
    assert grad(rows=0) == 0 and grad(cols=0) == 0 and grad(tokens=0, acc=1, out=None) == 0


def test_adapter_refusals(lib):
    def call(x=P, dtype=2, tokens=3, cols=8, ldx=8, a=P, b=P, adapters=2, rank=4, n=6, ids=P,
             base=None, ldb=6, out=P, odt=2, ldo=6):
        return lib.adapter_linear(x, dtype, tokens, cols, ldx, a, b, adapters, rank, n, ids, None,
                                  base, ldb, out, odt, ldo, None)
    _bad(lib, [lambda: call(dtype=0), lambda: call(dtype=3), lambda: call(odt=1),
               lambda: call(tokens=-1), lambda: call(tokens=1 << 24), lambda: call(cols=0),
               lambda: call(cols=(1 << 20) + 1), lambda: call(n=-1), lambda: call(n=(1 << 24) + 1),
               lambda: call(rank=0), lambda: call(rank=129), lambda: call(adapters=-1),
               lambda: call(adapters=8192), lambda: call(ldx=7), lambda: call(ldo=5),
               lambda: call(base=C.c_void_p(512), ldb=5), lambda: call(base=P, ldb=7),
               lambda: call(x=None), lambda: call(ids=None), lambda: call(out=None),
               lambda: call(a=None), lambda: call(b=None)])
    assert call(tokens=0) == 0 and call(n=0) == 0


def test_binding_refusals():
    """The binding checks shapes, types, strides and devices before the library is called."""
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    f = torch.zeros((6, 8))
    i = torch.zeros((6,), dtype=torch.int32)
    h = f.bfloat16()
    ad = torch.zeros((2, 4, 8), dtype=torch.bfloat16), torch.zeros((2, 5, 4), dtype=torch.bfloat16)
    for call in (lambda: B.beam_select(f, torch.zeros((2, 3)), 4),
                 lambda: B.beam_reorder(f, torch.zeros((2, 3), dtype=torch.int32)),
                 lambda: B.embedding_lookup(f, i), lambda: B.embedding_gradient(f, i, 5),
                 lambda: B.adapter_linear(h, *ad, i)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: B.beam_select(f.double(), torch.zeros((2, 3)), 4),
                 lambda: B.beam_select([[1.0]], torch.zeros((2, 3)), 4),
                 lambda: B.beam_reorder(f, [[0]]),
                 lambda: B.embedding_lookup(i, i), lambda: B.embedding_gradient(i, i, 4),
                 lambda: B.adapter_linear(i, *ad, i)):
        with pytest.raises(TypeError):
            call()


def test_state_layouts():
    """How the binding describes views: segments, dense tails, refused ones."""
    from approximate_nearest_neighbour_gb300 import binding as B
    assert B._dense_tail((4, 3, 5), (15, 5, 1)) == 1
    assert B._dense_tail((4, 3, 5), (30, 5, 1)) == 1
    assert B._dense_tail((4, 3, 5), (15, 1, 3)) == 3
    assert B._dense_tail((4, 3, 5), (40, 10, 1)) == 2
    assert B._dense_tail((4,), (1,)) == 1
    assert B._dense_tail((4, 3, 1), (3, 1, 7)) == 1
    assert B._segments((4, 3, 5), (40, 10, 1), 2, "t") == (3, 10)
    assert B._segments((4, 2, 3, 5), (60, 30, 10, 1), 3, "t") == (6, 10)
    with pytest.raises(ValueError):
        B._segments((4, 2, 3, 5), (99, 31, 10, 1), 3, "t")
