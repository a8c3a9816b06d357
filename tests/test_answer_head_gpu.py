"""The 4-bit head, the score adjustments, the k-selection and the distillation together."""

import importlib.util
import os

import numpy as np
import pytest

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


def test_decoding_follows_the_definitions(example):
    """Each step's token has the best adjusted score, up to fp32 rounding."""
    import torch
    head, states, xs = example.setup(rows=600, width=96)
    batch, steps = 5, 7
    tokens = example.decode(head, states, xs, batch=batch, steps=steps).cpu().numpy()
    assert (tokens % 2 == 0).all() and tokens.shape == (batch, steps)
    w = R.values(head.codes.cpu().numpy(), head.scales.cpu().numpy(), "nvfp4")[:, :96]
    w = w * float(head.scale)
    hist = np.full((batch, steps + 1), -1, np.int32)
    hist[:, 0] = np.arange(batch) * 7
    B = example.B
    for t in range(steps):
        x = states[torch.from_numpy(hist[:, t]).long().cuda()]
        qx = B.fp4_quantize(x, "nvfp4", tensor_scale=xs)
        v = R.values(qx[0].cpu().numpy(), qx[1].cpu().numpy(), "nvfp4")[:, :96] * float(xs)
        f = np.ones(batch)
        s, _ = R.adjust(v @ w.T, history=hist, history_len=np.full(batch, t + 1),
                        prompt_len=np.ones(batch, np.int32), repetition=1.3 * f, presence=0.5 * f,
                        frequency=0.5 * f, temperature=0.8 * f,
                        mask=np.full((1, 19), 0x55555555, np.int32))
        best = s.max(1)
        got = s[np.arange(batch), tokens[:, t]]
        assert (got >= best - 1e-4 * np.abs(best)).all()
        hist[:, t + 1] = tokens[:, t]


def test_the_student_learns(example):
    head, states, xs = example.setup(rows=512, width=64)
    losses = example.distill(head, states, xs, steps=40, batch=256, k=16).cpu().numpy()
    assert np.isfinite(losses).all() and losses[-1] < 0.5 * losses[0]
