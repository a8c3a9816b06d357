"""beam_reorder on views of unusual order: refused where they repeat memory, right elsewhere."""

import pytest

pytestmark = pytest.mark.gpu


def _reordered(t, beams):
    import torch
    groups, n = beams.shape
    rows = beams.long() + torch.arange(groups, device="cuda").unsqueeze(1) * n
    return t[rows.view(-1)]


@pytest.mark.parametrize("shape,stride", [
    ((4, 3, 5), (5, 5, 1)), ((4, 2, 5), (5, 10, 1)), ((6, 2, 5), (5, 25, 1)),
    ((4, 3, 5), (5, 15, 1))])
def test_repeated_memory_is_refused(shape, stride):
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    room = torch.arange(500, dtype=torch.float32, device="cuda")
    t = room.as_strided(shape, stride)
    beams = torch.zeros((1, shape[0]), dtype=torch.int32, device="cuda")
    for call in (lambda: B.beam_reorder(t, beams),
                 lambda: B.beam_reorder(torch.zeros(shape, device="cuda"), beams, out=t)):
        with pytest.raises(B.IVFPQError):
            call()
    assert torch.equal(room, torch.arange(500, dtype=torch.float32, device="cuda"))


@pytest.mark.parametrize("shape,stride", [
    ((4, 3, 5), (5, 20, 1)),     # rows inside segments: a buffer [3, 4, 5]
    ((4, 3, 5), (15, 5, 1)), ((4, 3, 5), (40, 7, 1)), ((4, 3, 5), (6, 100, 1)),
    ((4, 2, 5), (10, 25, 1)),    # neither inside the other
    ((4, 2, 5), (25, 10, 1)), ((4, 1, 5), (5, 0, 1)), ((4, 5, 3), (30, 6, 1))])
def test_any_order_of_rows_and_segments(shape, stride):
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    room = torch.arange(500, dtype=torch.float32, device="cuda")
    t = room.as_strided(shape, stride)
    beams = torch.tensor([[2, 2, 0, 3]], dtype=torch.int32, device="cuda")
    want = room.clone()
    want.as_strided(shape, stride).copy_(_reordered(t.clone(), beams))
    out = torch.full_like(room, -1.0)
    there = torch.full_like(room, -1.0)
    there.as_strided(shape, stride).copy_(_reordered(t.clone(), beams))
    B.beam_reorder(t, beams, out=out.as_strided(shape, stride))
    assert torch.equal(out, there)
    B.beam_reorder(t, beams)
    assert torch.equal(room, want)
