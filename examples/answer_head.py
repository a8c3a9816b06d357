"""A 4-bit output head that answers, and a smaller student that learns from its top lists.

    python examples/answer_head.py

Runs the 4-bit product, the score adjustments, the k-selection and the distillation as
they are used together:

* the teacher's table of 4,096 rows is quantized once (NVFP4);
* decode(): one token at a time, fp4_linear makes the scores of every row of a batch,
  score_adjust applies repetition penalties, a temperature and a mask of allowed rows
  and negates them, kselect takes the best, which become the next tokens;
* search(): the same with beams and requests' own adapters: embedding_lookup takes the
  tokens' states, adapter_linear adds each request's low-rank adapter to the shared scores,
  beam_select takes the best continuations, beam_reorder moves the histories to them;
* distill(): the teacher's top list of each state (kselect's values and ids) trains a
  student head with topk_distill.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from approximate_nearest_neighbour_gb300 import binding as B  # noqa: E402


class Head:
    """A [rows, width] table in 4-bit form."""

    def __init__(self, table, fmt="nvfp4"):
        self.fmt = fmt
        self.rows = table.shape[0]
        # the tensor's scale puts its largest magnitude at E4M3 x E2M1's largest
        self.scale = (table.abs().amax().float() / (448.0 * 6.0)).view(1)
        self.codes, self.scales = B.fp4_quantize(table, fmt, tensor_scale=self.scale)

    def scores(self, x, x_scale, dtype=torch.float32):
        return B.fp4_linear(x, self.codes, self.scales, self.fmt, x_tensor_scale=x_scale,
                            w_tensor_scale=self.scale, dtype=dtype)


def setup(rows=4096, width=256, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.randn((rows, width), generator=gen, device="cuda") * width ** -0.5
    states = torch.randn((rows, width), generator=gen, device="cuda", dtype=torch.float32)
    x_scale = (states.abs().amax() / (448.0 * 6.0)).view(1)
    return Head(table), states.to(torch.bfloat16), x_scale


def decode(head, states, x_scale, batch=8, steps=16, k=4):
    """Tokens [batch, steps]: each step's state is that of the last token."""
    device = states.device
    history = torch.full((batch, steps + 1), -1, dtype=torch.int32, device=device)
    history[:, 0] = torch.arange(batch, device=device) * 7
    length = torch.ones((batch,), dtype=torch.int32, device=device)
    prompt = torch.ones_like(length)
    flat = torch.full((batch,), 1.0, device=device)
    # only even rows may be answered
    mask = torch.full((1, (head.rows + 31) // 32), 0x55555555, dtype=torch.int32, device=device)
    for t in range(steps):
        x = states[history[:, t].long()]
        scores = head.scores(x, x_scale)
        cost = B.score_adjust(scores, history=history, history_len=length, prompt_len=prompt,
                              repetition=1.3 * flat, presence=0.5 * flat, frequency=0.5 * flat,
                              temperature=0.8 * flat, mask=mask, negate=True, out=scores)
        _, ids = B.kselect(cost, k)
        history[:, t + 1] = ids[:, 0].int()
        length += 1
    return history[:, 1:]


def adapters(head, width, count=3, rank=8, seed=1):
    """Low-rank adapters [count, rank, width] and [count, rows, rank], and their scales."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randn((count, rank, width), generator=gen, device="cuda") * width ** -0.5
    b = torch.randn((count, head.rows, rank), generator=gen, device="cuda") * 0.2
    return a.bfloat16(), b.bfloat16(), torch.full((count,), 0.5, device="cuda")


def search(head, states, x_scale, low_rank, requests=3, beams=4, steps=8, end=0):
    """(tokens [requests, beams, steps], totals [requests, beams]), best beams first;
    request i has adapter i - 1, the first one none; a beam ends with the token `end`."""
    device = states.device
    a, b, scales = low_rank
    rows = requests * beams
    which = (torch.arange(rows, device=device) // beams - 1).int()
    history = torch.zeros((rows, steps + 1), dtype=torch.int32, device=device)
    history[:, 0] = (torch.arange(rows, device=device) // beams * 7 + 3).int()
    totals = torch.full((requests, beams), -float("inf"), device=device)
    totals[:, 0] = 0.0  # all beams are alike at first: one is enough
    finished = torch.zeros((requests, beams), dtype=torch.bool, device=device)
    length = torch.ones((requests,), dtype=torch.int32, device=device)
    heat = torch.full((rows,), 0.7, device=device)
    for t in range(steps):
        x = B.embedding_lookup(states, history[:, t].contiguous())
        scores = head.scores(x, x_scale)
        B.adapter_linear(x, a, b, which, scales=scales, base=scores, out=scores)
        B.score_adjust(scores, temperature=heat, out=scores)
        totals, of, ids = B.beam_select(scores, totals, beams, finished=finished, end_id=end)
        B.beam_reorder(history, of, lengths=length)
        finished = finished.gather(1, of.clamp(min=0).long()) | (ids == end)
        history[:, t + 1] = ids.view(-1)
        length += 1
    return history[:, 1:].view(requests, beams, steps), totals


def distill(head, states, x_scale, steps=60, batch=512, k=32, tau=2.0, rate=30.0):
    """The mean loss before each step of a student head learning the teacher's lists."""
    student = torch.zeros((head.rows, states.shape[1]), device=states.device)
    weight = torch.full((batch,), 1.0 / batch, device=states.device)
    losses = []
    for t in range(steps):
        x = states[(torch.arange(batch, device=states.device) * 5 + t * batch) % head.rows]
        vals, ids = B.kselect(-head.scores(x, x_scale) * 4.0, k)  # ascending costs: t = -value
        scores = x.float() @ student.t()
        # the gradient takes the scores' place
        loss, grad = B.topk_distill(scores, vals, ids, weight, tau, negated=True, grad=scores)
        student -= rate * (grad.t() @ x.float())
        losses.append(loss.mean())
    return torch.stack(losses)


def main():
    head, states, x_scale = setup()
    tokens = decode(head, states, x_scale)
    losses = distill(head, states, x_scale)
    beams, totals = search(head, states, x_scale, adapters(head, states.shape[1]))
    B.device_check()
    print("tokens of the first rows:", tokens[:2].tolist())
    print("best beam of each request:", beams[:, 0].tolist(), totals[:, 0].tolist())
    print("distillation loss: %.4f -> %.4f" % (float(losses[0]), float(losses[-1])))


if __name__ == "__main__":
    main()
