"""beam_reorder with states that hold nothing, beside others."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape,axis", [((6, 0, 5), 2), ((6, 0, 5), 1), ((6, 4, 0), 1),
                                        ((6, 0, 3, 8), 2), ((6, 0, 0), 1)])
@pytest.mark.parametrize("lengths", [True, False])
@pytest.mark.parametrize("in_place", [True, False])
def test_empty_states(shape, axis, lengths, in_place):
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    beams = torch.tensor([[1, 1, 0], [2, 0, 0]], dtype=torch.int32, device="cuda")
    n = torch.tensor([2, 4], dtype=torch.int32, device="cuda") if lengths else None
    t = torch.randn((6, 4), device="cuda")
    rows = (beams.long() + torch.tensor([[0], [3]], device="cuda")).view(-1)
    want = t[rows]
    if lengths:
        want = torch.cat([want[:, :2], torch.stack([t[:3, 2:], want[3:, 2:]]).view(6, 2)], 1)
    states = [torch.zeros(shape, device="cuda"), t.clone(), torch.zeros(shape, device="cuda")]
    out = None if in_place else [torch.zeros(shape, device="cuda"), t.clone(),
                                 torch.zeros(shape, device="cuda")]
    got = B.beam_reorder(states, beams, lengths=n, axis=[axis, 1, axis], out=out)
    assert torch.equal(got[1], want)
