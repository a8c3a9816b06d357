"""score_adjust with the longest history the interface takes."""

import pytest

pytestmark = pytest.mark.gpu


def test_the_longest_history():
    """2^31 - 1 tokens: the step past the last one stays inside 32 bits. (The bias list's
    loop counts the same way; a list that long would keep one block busy for seconds.)"""
    import torch
    from approximate_nearest_neighbour_gb300 import binding as B
    n = 2**31 - 1
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 10 GB")
    h = torch.full((1, n), -1, dtype=torch.int32, device="cuda")
    h[0, 0] = 3
    h[0, n - 1] = 3
    h[0, n - 300] = 5
    h[0, n - 2000] = 63
    x = torch.full((1, 64), 10.0, device="cuda")
    f = torch.ones((1,), device="cuda")
    prompt = torch.tensor([n - 1000], dtype=torch.int32, device="cuda")
    got = B.score_adjust(x, history=h, prompt_len=prompt, repetition=2 * f, frequency=f,
                         presence=0.5 * f)
    want = torch.full((1, 64), 10.0)
    # 10 / 2, less one count and the presence penalty past the prompt
    want[0, 3], want[0, 5], want[0, 63] = 3.5, 3.5, 5.0
    assert torch.equal(got.cpu(), want)
