"""embedding_lookup and embedding_gradient do not write over what they read."""

import pytest

pytestmark = pytest.mark.gpu


def test_outputs_have_memory_of_their_own():
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    t = torch.randn((12, 16), device="cuda")
    keep = t.clone()
    ids = torch.arange(11, -1, -1, dtype=torch.int32, device="cuda")
    for call in (lambda: B.embedding_lookup(t, ids, out=t),
                 lambda: B.embedding_lookup(t, ids.view(3, 4), out=t.view(3, 4, 16)),
                 lambda: B.embedding_lookup(t, ids[:5], out=t[:5]),
                 lambda: B.embedding_gradient(t, ids, 12, out=t),
                 lambda: B.embedding_gradient(t, ids, 5, out=t[:5], accumulate=True)):
        with pytest.raises(ValueError, match="memory"):
            call()
    assert torch.equal(t, keep)
    # columns of one buffer beside each other are
    both = torch.zeros((12, 32), device="cuda")
    both[:, :16] = t
    B.embedding_lookup(both[:, :16], ids, out=both[:, 16:])
    assert torch.equal(both[:, 16:], t.flip(0)) and torch.equal(both[:, :16], t)
    B.embedding_gradient(both[:, :16], ids, 12, out=both[:, 16:])
    assert torch.equal(both[:, 16:], t.flip(0))
    none = torch.zeros((0, 16), device="cuda")
    assert B.embedding_lookup(none, ids[:0], out=none) is none
