"""Sizes at the ends of their types are refused before anything is computed from them."""

import ctypes as C

import pytest

P = C.c_void_p(256)


@pytest.fixture(scope="module")
def lib():
    from approximate_nearest_neighbour_gb300 import binding, build
    build.build_library()
    return binding.lib()


@pytest.mark.parametrize("groups", [1 << 31, 1 << 57, 1 << 58, 1 << 62, (1 << 63) - 1])
@pytest.mark.parametrize("beams", [1, 3, 4, 64])
def test_groups_of_beams(lib, groups, beams):
    from approximate_nearest_neighbour_gb300 import binding as B
    assert lib.beam_select(P, 0, groups, beams, 8, 8, P, None, 0, 4, P, P, P,
                           None) == B.IVFPQ_ERR_INVALID_ARG
    assert b"groups=%d" % groups in lib.ivfpq_last_error()
