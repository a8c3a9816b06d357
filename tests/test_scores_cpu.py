"""Host-side refusals of the 4-bit, score-adjustment and distillation entry points."""

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


def test_fp4_refusals(lib):
    p, odd = C.c_void_p(256), C.c_void_p(257)
    _bad(lib, [
        lambda: lib.fp4_quantize(p, 3, 4, 32, 32, 0, None, p, p, None),       # element type
        lambda: lib.fp4_quantize(p, 0, 4, 32, 32, 2, None, p, p, None),       # format
        lambda: lib.fp4_quantize(p, 0, -1, 32, 32, 0, None, p, p, None),      # rows
        lambda: lib.fp4_quantize(p, 0, 4, 0, 32, 0, None, p, p, None),        # cols
        lambda: lib.fp4_quantize(p, 0, 4, 32, 31, 0, None, p, p, None),       # overlapping rows
        lambda: lib.fp4_quantize(None, 0, 4, 32, 32, 0, None, p, p, None),    # null
        lambda: lib.fp4_quantize(p, 0, 4, 32, 32, 0, None, odd, p, None),     # alignment
        lambda: lib.fp4_dequantize(p, p, 4, 32, 7, None, p, 0, None),
        lambda: lib.fp4_dequantize(p, p, 4, 32, 0, None, p, -1, None),
        lambda: lib.fp4_dequantize(p, None, 4, 32, 0, None, p, 0, None),
        lambda: lib.fp4_product(p, p, 4, p, p, 4, 0, 0, None, None, p, 0, None),
        lambda: lib.fp4_product(p, p, -4, p, p, 4, 32, 0, None, None, p, 0, None),
        lambda: lib.fp4_product(p, p, 1 << 24, p, p, 4, 32, 0, None, None, p, 0, None),
        lambda: lib.fp4_product(p, p, 4, p, p, 1 << 31, 32, 0, None, None, p, 0, None),
        lambda: lib.fp4_product(p, p, 4, p, p, 4, 32, 0, None, None, p, 9, None),
        lambda: lib.fp4_product(p, p, 4, p, p, 4, 32, 0, None, None, None, 0, None),
        lambda: lib.fp4_product(odd, p, 4, p, p, 4, 32, 0, None, None, p, 0, None),
        lambda: lib.fp4_linear(p, 5, 4, 32, p, p, 4, 32, 0, None, None, p, 0, None),
        lambda: lib.fp4_linear(p, 0, 4, 16, p, p, 4, 32, 0, None, None, p, 0, None),
        lambda: lib.fp4_linear(p, 0, 4, 32, p, odd, 4, 32, 0, None, None, p, 0, None),
    ])
    assert lib.fp4_quantize(None, 0, 0, 32, 32, 0, None, None, None, None) == 0
    assert lib.fp4_product(None, None, 0, p, p, 4, 32, 0, None, None, None, 0, None) == 0


def test_adjust_refusals(lib):
    p = C.c_void_p(256)

    def call(scores=p, dtype=0, rows=2, cols=8, lds=8, history=None, hl=None, bi=None, bv=None,
             out=p, odt=0, ldo=8):
        return lib.score_adjust(scores, dtype, rows, cols, lds, history, 4, 4, hl, None, None, None,
                                None, bi, bv, 1, None, None, 0, 0, out, odt, ldo, None)

    _bad(lib, [lambda: call(dtype=4), lambda: call(rows=-1), lambda: call(cols=-1),
               lambda: call(cols=1 << 29), lambda: call(lds=7), lambda: call(ldo=7),
               lambda: call(scores=None), lambda: call(out=None), lambda: call(hl=p),
               lambda: call(bi=p), lambda: call(bv=p), lambda: call(odt=1),
               lambda: call(dtype=2, odt=1)])
    assert call(rows=0) == 0 and call(cols=0) == 0


def test_distill_refusals(lib):
    p = C.c_void_p(256)
    fwd, bwd, both = lib.topk_distill_forward, lib.topk_distill_backward, lib.topk_distill
    _bad(lib, [
        lambda: fwd(p, 3, 2, 8, 8, p, p, 2, 1.0, 0, p, p, None),
        lambda: fwd(p, 0, 2, 0, 8, p, p, 2, 1.0, 0, p, p, None),
        lambda: fwd(p, 0, 2, 8, 7, p, p, 2, 1.0, 0, p, p, None),
        lambda: fwd(p, 0, 2, 8, 8, p, p, 0, 1.0, 0, p, p, None),
        lambda: fwd(p, 0, 2, 8, 8, p, p, 2049, 1.0, 0, p, p, None),
        lambda: fwd(p, 0, 2, 8, 8, p, p, 2, 0.0, 0, p, p, None),
        lambda: fwd(p, 0, 2, 8, 8, p, p, 2, float("nan"), 0, p, p, None),
        lambda: fwd(p, 0, 2, 8, 8, p, p, 2, float("inf"), 0, p, p, None),
        lambda: fwd(p, 0, 2, 8, 8, p, p, 2, 1.0, 0, None, p, None),
        lambda: bwd(p, 0, 2, 8, 8, p, p, 2, 1.0, 0, p, p, p, 7, None),
        lambda: bwd(p, 0, 2, 8, 8, p, p, 2, -1.0, 0, p, p, p, 8, None),
        lambda: bwd(p, 0, 2, 8, 8, p, p, 2, 1.0, 0, p, None, p, 8, None),
        lambda: both(p, 0, 2, 8, 8, p, p, 2, 1.0, 0, p, None, p, 8, None),
        lambda: both(p, 0, 2, 8, 8, p, p, 2, 1.0, 0, p, p, p, 7, None),
        lambda: both(p, 0, -2, 8, 8, p, p, 2, 1.0, 0, p, p, p, 8, None),
    ])
    assert fwd(None, 0, 0, 8, 8, None, None, 2, 1.0, 0, None, None, None) == 0


def test_binding_refusals():
    """The binding checks shapes, types, strides and devices before the library is called."""
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    f, u8, i32, i64 = (lambda *s, t=t: torch.zeros(s, dtype=t, device="meta")
                       for t in (torch.float32, torch.uint8, torch.int32, torch.int64))
    cpu = torch.zeros((2, 64))
    for call in (lambda: B.fp4_quantize(cpu), lambda: B.score_adjust(cpu),
                 lambda: B.topk_distill_forward(cpu, cpu, torch.zeros((2, 64), dtype=torch.int64)),
                 lambda: B.fp4_dequantize(torch.zeros((2, 32), dtype=torch.uint8), u8(1, 1, 512))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: B.fp4_quantize(torch.zeros((2, 64), dtype=torch.float64)),
                 lambda: B.fp4_quantize([[1.0]]),
                 lambda: B.score_adjust(i32(2, 3))):
        with pytest.raises(TypeError):
            call()
    for fmt in ("fp4", 2, None):
        with pytest.raises(ValueError):
            B.fp4_shapes(1, 1, fmt)


def test_packed_shapes():
    from approximate_nearest_neighbour_gb300 import binding as B
    assert B.fp4_shapes(1, 1) == ((1, 16), (1, 1, 512))
    assert B.fp4_shapes(129, 129) == ((129, 80), (2, 2, 512))
    assert B.fp4_shapes(128, 96, "nvfp4") == ((128, 48), (1, 2, 512))
    assert B.fp4_shapes(0, 64, "nvfp4") == ((0, 32), (0, 1, 512))
