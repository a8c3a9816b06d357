"""beam_reorder with lengths beyond any state, and positions of gigabytes."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [5, 64])
def test_lengths_past_the_positions(size):
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    t = torch.randn((6, 3, 20, size), device="cuda")
    beams = torch.tensor([[1, 1, 0], [2, 0, 0]], dtype=torch.int32, device="cuda")
    rows = (beams.long() + torch.tensor([[0], [3]], device="cuda")).view(-1)
    for n in (20, 21, 1 << 30, 2 ** 31 - 1):
        lengths = torch.full((2,), n, dtype=torch.int32, device="cuda")
        mine = t.clone()
        B.beam_reorder(mine, beams, lengths=lengths, axis=2)
        assert torch.equal(mine, t[rows])
    mine = t.clone()
    B.beam_reorder(mine, beams, lengths=torch.full((2,), -2 ** 31, dtype=torch.int32,
                                                   device="cuda"), axis=2)
    assert torch.equal(mine, t)


def test_positions_of_gigabytes():
    """A length of 2^31 - 1 times a position of 2^32 + 16 bytes."""
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 9 GB")
    size = (1 << 32) + 16
    t = torch.zeros((2, 1, size), dtype=torch.uint8, device="cuda")
    t[1, 0, :50] = 3
    t[1, 0, -50:] = 4
    beams = torch.tensor([[1, 1]], dtype=torch.int32, device="cuda")
    B.beam_reorder(t, beams, lengths=torch.tensor([2 ** 31 - 1], dtype=torch.int32, device="cuda"))
    assert (t[:, 0, :50] == 3).all() and (t[:, 0, -50:] == 4).all()
    assert int(t[:, 0, 1000:-1000].max()) == 0
