"""Lookup, shared 4-bit product, adapters, adjustment, beam selection and reordering in a row."""

import importlib.util
import os

import numpy as np
import pytest

import decode_ref as D
import scores_ref as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "answer_head", os.path.join(ROOT, "examples", "answer_head.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _values(head, x, x_scale, B):
    """fp64 scores of the 4-bit product."""
    w = R.values(head.codes.cpu().numpy(), head.scales.cpu().numpy(), "nvfp4")[:, :x.shape[1]]
    q = B.fp4_quantize(x, "nvfp4", tensor_scale=x_scale)
    v = R.values(q[0].cpu().numpy(), q[1].cpu().numpy(), "nvfp4")[:, :x.shape[1]]
    return (v * float(x_scale)) @ (w * float(head.scale)).T


def test_search_follows_the_definitions(example):
    """Replays the search in fp64: every beam's total is that of its tokens, and no
    continuation that was left out is better than the worst one taken, up to the error
    of fp32 scores (sums of 96 products and of 8; 2^-24 each of magnitudes below 64)
    accumulated over the steps."""
    import torch
    head, states, xs = example.setup(rows=600, width=96)
    a, b, scales = example.adapters(head, 96)
    requests, beams, steps = 3, 4, 6
    tokens, totals = example.search(head, states, xs, (a, b, scales), requests, beams, steps)
    example.B.device_check()
    tokens, totals = tokens.cpu().numpy(), totals.double().cpu().numpy()
    tol = 1e-4 * steps
    assert (np.diff(totals, axis=1) <= 0).all()
    for r in range(requests):
        # a plain search over the same scores
        live = [((r * 7 + 3,), 0.0, False)]
        for t in range(steps):
            every = []
            for path, total, done in live:
                if done:
                    every.append((total, path + (0,), True))
                    continue
                x = states[path[-1]:path[-1] + 1]
                s = _values(head, x, xs, example.B)
                x64 = x.double().cpu().numpy()
                s, _, _ = D.adapter(x64, a.double().cpu().numpy(), b.double().cpu().numpy(), [r - 1],
                                    scales.double().cpu().numpy(), s)
                lp = D.log_softmax(s[0] / np.float32(0.7)) + total
                for c in np.argsort(-lp)[:beams]:
                    every.append((lp[c], path + (int(c),), c == 0))
            every.sort(key=lambda e: -e[0])
            live = [(p, v, d) for v, p, d in every[:beams]]
        want = np.array([v for _, v, _ in live])
        assert (np.abs(totals[r] - want) <= tol + 1e-5 * np.abs(want)).all(), (totals[r], want)
        gap = np.abs(np.diff(want)).min() if beams > 1 else 1.0
        if gap > 2 * tol:  # the order is beyond rounding
            assert [tuple(v) for v in tokens[r].tolist()] == [p[1:] for p, _, _ in live]


def test_search_is_captured(example):
    """One step of the search in a graph, replayed on other states."""
    import torch
    B = example.B
    head, states, xs = example.setup(rows=512, width=64)
    a, b, scales = example.adapters(head, 64)
    ids = torch.arange(8, dtype=torch.int32, device="cuda")
    which = torch.tensor([-1, -1, 0, 0, 1, 1, 2, 2], dtype=torch.int32, device="cuda")
    totals = torch.zeros((4, 2), device="cuda")
    cache = torch.randn((8, 3, 20, 16), device="cuda").bfloat16()
    length = torch.tensor([5, 20, 1, 11], dtype=torch.int32, device="cuda")

    def step(cache):
        x = B.embedding_lookup(states, ids, 0.5)
        s = head.scores(x, xs)
        B.adapter_linear(x, a, b, which, scales=scales, base=s, out=s)
        out = B.beam_select(s, totals, 2)
        B.beam_reorder(cache, out[1], lengths=length, axis=2)
        return out

    step(cache.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(cache)
    for first in (3, 100, 250):
        ids.copy_(torch.arange(first, first + 8, device="cuda"))
        other = cache.clone()
        graph.replay()
        want = step(other)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want)) and torch.equal(cache, other)
