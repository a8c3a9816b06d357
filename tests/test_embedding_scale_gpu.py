"""embedding_lookup with scales that are not finite or negative."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [float("inf"), -float("inf"), float("nan"), -2.0, 0.0])
@pytest.mark.parametrize("name,out", [("float32", "float32"), ("bfloat16", "bfloat16"),
                                      ("float16", "float32")])
@pytest.mark.parametrize("cols", [64, 65])
def test_ids_outside_give_zeros(scale, name, out, cols):
    """Whole vectors and rows at odd offsets: +0 outside the table, the product inside."""
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    table = torch.randn((9, cols), device="cuda").to(getattr(torch, name))
    ids = torch.tensor([3, -1, 9, 0, 2 ** 31 - 1, 8], dtype=torch.int32, device="cuda")
    got = B.embedding_lookup(table, ids, scale, dtype=getattr(torch, out))
    inside = [0, 3, 5]
    want = (table[ids[inside].long()].float() * scale).to(got.dtype)
    assert torch.equal(got[inside].isnan(), want.isnan())
    assert torch.equal(got[inside].nan_to_num(), want.nan_to_num())
    outside = got[[1, 2, 4]]
    assert (outside == 0).all() and not torch.signbit(outside).any()
