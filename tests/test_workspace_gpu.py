"""Calls that take workspace, in programs that wait after each call."""

import time

import pytest

pytestmark = pytest.mark.gpu


def _waited(fn, n=100, rounds=5):
    """Microseconds of fn with a synchronisation after it: the least of a few means."""
    import torch
    best = float("inf")
    for _ in range(rounds):
        fn()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            fn()
            torch.cuda.synchronize()
        best = min(best, (time.perf_counter() - t) / n * 1e6)
    return best


def test_workspace_outlives_a_wait():
    """One token through a layer with a wait after it, as decoding does to read the
    token: the one call costs no more than twice its two halves, which take none."""
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((1, 4096), generator=gen, device="cuda", dtype=torch.float32).bfloat16()
    w = B.fp4_quantize(torch.randn((4096, 4096), generator=gen, device="cuda"))
    q = B.fp4_quantize(x)
    out = torch.empty((1, 4096), dtype=torch.bfloat16, device="cuda")

    def halves():
        B.fp4_quantize(x, codes=q[0], scales=q[1])
        B.fp4_product(*q, *w, out=out)

    two = _waited(halves)
    one = _waited(lambda: B.fp4_linear(x, *w, out=out))
    assert one <= 2 * two


def test_calls_of_several_streams_and_a_captured_one():
    """Workspace in use on one stream is not given to another, and a captured call has its own."""
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = B.fp4_quantize(torch.randn((6000, 4096), generator=gen, device="cuda"))
    xs = [torch.randn((m, 4096), generator=gen, device="cuda") for m in (1, 40, 300, 2000)]
    want = [B.fp4_linear(x, *w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(20):
        got = [B.fp4_linear(x, *w, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = xs[1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = B.fp4_linear(x, *w)
    for other in (xs[1], xs[1].flip(0)):
        x.copy_(other)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, B.fp4_linear(other, *w))
