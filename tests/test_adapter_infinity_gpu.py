"""adapter_linear with infinities and NaN among its operands: the definition's, and in no
other token's row."""

import pytest

pytestmark = pytest.mark.gpu


def _case(tokens, rank, dtype, out):
    """Operands above zero, so that no infinity meets a zero or another sign."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(tokens + rank)
    ru = lambda *s: torch.rand(s, generator=g, device="cuda") * 0.5 + 0.25  # noqa: E731
    dt, cols, n = getattr(torch, dtype), 72, 40
    ids = (torch.arange(tokens, device="cuda") % 3 - 1).int()  # a third without an adapter
    return dict(x=ru(tokens, cols).to(dt), a=ru(2, rank, cols).to(dt), b=ru(2, n, rank).to(dt),
                ids=ids, scales=torch.ones(2, device="cuda"),
                base=ru(tokens, n).to(getattr(torch, out)))


def _want(x, a, b, ids, scales, base):
    import torch
    y = base.double()
    for i in range(a.shape[0]):
        t = ids == i
        y[t] += scales[i].double() * (x[t].double() @ a[i].double().T @ b[i].double().T)
    return y


def _same(got, want):
    """The same NaN and infinities; how near finite results are is tested elsewhere."""
    import torch
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.isposinf(), want.isposinf())
    assert torch.equal(got.isneginf(), want.isneginf())


@pytest.mark.parametrize("dtype,out", [("float16", "float16"), ("bfloat16", "bfloat16"),
                                       ("float16", "float32"), ("bfloat16", "float32")])
@pytest.mark.parametrize("tokens", [9, 70, 300])
@pytest.mark.parametrize("rank", [1, 3, 4, 8, 9, 16, 24, 40, 72, 100, 128])
def test_infinite_inputs(dtype, out, tokens, rank):
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    c = _case(tokens, rank, dtype, out)
    clean = B.adapter_linear(**c)
    rows = {1: float("inf"), 2: -float("inf"), 4: float("nan"), 3: float("inf")}  # 3: no adapter
    for t, v in rows.items():
        c["x"][t, 5] = v
    got, want = B.adapter_linear(**c), _want(**c)
    assert want[1].isposinf().all() and want[2].isneginf().all() and want[3].isfinite().all()
    _same(got, want)
    others = [t for t in range(tokens) if t not in (1, 2, 4)]
    assert torch.equal(got[others], clean[others])


@pytest.mark.parametrize("out", ["float16", "float32"])
@pytest.mark.parametrize("tokens", [9, 300])
def test_an_infinite_element_beside_large_ones(out, tokens):
    """fp16: of a token's x A^T one element is infinite, another past fp16's range."""
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    c = _case(tokens, 8, "float16", out)
    c["a"][:, 0, 3] = float("inf")
    c["a"][:, 1] = -6e4  # about -1e6 after the product
    got, want = B.adapter_linear(**c), _want(**c)
    t = c["ids"] >= 0
    assert want[t].isposinf().all()
    _same(got, want)
