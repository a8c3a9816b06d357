"""beam_reorder refuses states whose written segments meet one another."""

import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from approximate_nearest_neighbour_gb300 import binding, build
    build.build_library()
    return binding.lib()


@pytest.mark.parametrize("rows,row,outer,step,inner", [
    (4, 20, 3, 20, 20),      # rows and segments one after the other in the same places
    (4, 20, 2, 40, 20), (4, 40, 3, 20, 20), (2, 60, 4, 20, 20), (6, 20, 2, 100, 20),
    (4, 40, 2, 100, 21),     # the second segment ends inside the fourth row
    (3, 30, 3, 45, 20), (4, 1000, 6, 30, 31), (2, 0, 1, 0, 4), (2, 64, 2, 0, 4),
    (4, 1 << 56, 2, 64, 64), (4, 64, 2, 1 << 60, 64)])
@pytest.mark.parametrize("in_place", [True, False])
def test_refused(lib, rows, row, outer, step, inner, in_place):
    from approximate_nearest_neighbour_gb300 import binding as B
    a = (C.c_int64 * B._STATE)(256 if in_place else 1 << 40, 256, row, row, outer, step, step,
                               inner, 0)
    rc = lib.beam_reorder(a, 1, C.c_void_p(4096), 1, rows, rows, None, None)
    assert rc == B.IVFPQ_ERR_INVALID_ARG
    assert b"beam_reorder: state 0" in lib.ivfpq_last_error()
