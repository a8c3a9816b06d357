"""Cases for the 4-bit block-scaled, score-adjustment and top-k distillation operators.

Each case is one call (or the short run of calls that belongs together) as a user of
the library makes it:

* quantize        vectors to 4-bit blocks, read back as the values they stand for
* product         scores of 4-bit queries against a 4-bit table, fp32 for a k-selection
* linear          floating activations through a 4-bit weight matrix
* adjust          penalties, biases, temperature and a bit mask on score rows
* distill_forward   a student's loss against a teacher's top list
* distill_backward  its gradient, from the forward's row statistics
* distill           both in one call, as a training step makes it

The plain forms are elementary torch operations in fp32; `exact` restates the same
definitions in fp64.
"""

import math

import torch

own = False


DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def _binding():
    from approximate_nearest_neighbour_gb300 import binding
    return binding


# ---------------------------------------------------------------------------
# cases
def listed():
    return [
        # one token's activations of a 4,096-wide layer, before its 4-bit product
        {"name": "quantize one token", "op": "quantize", "fmt": "mxfp4", "dtype": "bf16",
         "rows": 1, "cols": 4096},
        # a batch of 10,000 queries of 128 dimensions, as the flat search takes them
        {"name": "quantize queries", "op": "quantize", "fmt": "nvfp4", "dtype": "f32",
         "rows": 10000, "cols": 128},
        # a vocabulary-sized weight matrix laid out once (odd row count)
        {"name": "quantize table", "op": "quantize", "fmt": "mxfp4", "dtype": "bf16",
         "rows": 65537, "cols": 4096},
        # 10,000 queries against 65,536 centroids of 96 dimensions: the large coarse pass
        {"name": "product coarse", "op": "product", "fmt": "nvfp4", "dtype": "f32",
         "rows": 10000, "n": 65536, "cols": 96},
        # a small batch of queries against an odd number of vectors
        {"name": "product ragged", "op": "product", "fmt": "mxfp4", "dtype": "f32",
         "rows": 77, "n": 100003, "cols": 128},
        # one decoded token through an output head
        {"name": "linear one token", "op": "linear", "fmt": "mxfp4", "dtype": "bf16",
         "rows": 1, "n": 32000, "cols": 4096},
        # a decoding batch of odd size through a wide layer
        {"name": "linear 37 tokens", "op": "linear", "fmt": "nvfp4", "dtype": "bf16",
         "rows": 37, "n": 16384, "cols": 4096},
        # a whole prompt batch through the same layer: the compute-bound end
        {"name": "linear prompt", "op": "linear", "fmt": "nvfp4", "dtype": "bf16",
         "rows": 8192, "n": 16384, "cols": 4096},
        # one request's scores with a short history: latency
        {"name": "adjust one request", "op": "adjust", "dtype": "f32", "rows": 1, "cols": 32000,
         "hist": 200, "nb": 8, "mask": "none", "negate": True},
        # a serving batch with long histories, biases and a grammar mask
        {"name": "adjust batch", "op": "adjust", "dtype": "bf16", "rows": 256, "cols": 131072,
         "hist": 4096, "nb": 64, "mask": "rows", "negate": False},
        # an odd, small evaluation batch: loss only
        {"name": "distill forward", "op": "distill_forward", "dtype": "f32", "rows": 37,
         "cols": 32001, "k": 10, "temperature": 1.0},
        # a training step over a vocabulary: loss and gradient
        {"name": "distill step", "op": "distill", "dtype": "bf16", "rows": 2048, "cols": 65536,
         "k": 100, "temperature": 2.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "linear", "adjust", "distill_forward",
                     "distill_backward", "distill"])
    if op == "quantize":
        cols = _log(rng, 48, 8192)
        return {"op": op, "fmt": rng.choice(["mxfp4", "nvfp4"]),
                "dtype": rng.choice(["f32", "f16", "bf16"]),
                "rows": _log(rng, 1, min(65537, 120_000_000 // cols)), "cols": cols}
    if op == "product":
        cols = rng.choice([64, 96, 128, _log(rng, 32, 768)])
        n = _log(rng, 200, 262144)
        return {"op": op, "fmt": rng.choice(["mxfp4", "nvfp4"]), "dtype": "f32",
                "rows": _log(rng, 1, min(10000, 500_000_000 // n)), "n": n, "cols": cols}
    if op == "linear":
        cols = _log(rng, 256, 8192)
        n = _log(rng, 256, min(65536, 200_000_000 // cols))
        return {"op": op, "fmt": rng.choice(["mxfp4", "nvfp4"]),
                "dtype": rng.choice(["f16", "bf16"]),
                "rows": _log(rng, 1, min(8192, 400_000_000_000 // (n * cols))), "n": n,
                "cols": cols}
    cols = _log(rng, 1000, 200_000)
    if op == "adjust":
        return {"op": op, "dtype": rng.choice(["f32", "f16", "bf16"]),
                "rows": _log(rng, 1, min(512, 30_000_000 // cols)), "cols": cols,
                "hist": _log(rng, 1, 8192), "nb": rng.choice([0, 1, 16, 300]),
                "mask": rng.choice(["none", "one", "rows"]), "negate": rng.random() < 0.5}
    return {"op": op, "dtype": rng.choice(["f32", "f16", "bf16"]),
            "rows": _log(rng, 1, min(4096, 60_000_000 // cols)), "cols": cols,
            "k": _log(rng, 1, min(1000, cols // 2)),
            "temperature": rng.choice([0.5, 1.0, 2.0, 4.0])}


# ---------------------------------------------------------------------------
# the 4-bit formats in plain torch
def _pow2(e):
    """2^e for int32 e in [-127, 127], exactly."""
    return ((e + 1 + 127).clamp(1, 254).to(torch.int32) << 23).view(torch.float32) * 0.5


def _round_e2m1(y):
    """Nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 in magnitude, ties to the even code, saturating."""
    a = y.abs().clamp(max=6.0)
    r = torch.where(a < 2, (a * 2).round() * 0.5, torch.where(a < 4, a.round(), (a * 0.5).round() * 2))
    return torch.copysign(r, y)


def _blocks(x, block):
    """x [rows, cols] in fp32, zero-padded to whole 32-column groups, as [rows, nblk, block]."""
    rows, cols = x.shape
    kp = -(-cols // 32) * 32
    x = x.float()
    if kp != cols:
        x = torch.nn.functional.pad(x, (0, kp - cols))
    return x.view(rows, kp // block, block)


def _quantize(x, fmt, g):
    """(element values [rows, nblk, block], scale bytes uint8 [rows, nblk], scale values)."""
    b = _blocks(x, BLOCK[fmt])
    amax = b.abs().amax(-1)
    if fmt == "mxfp4":
        _, ex = torch.frexp(amax)
        e = torch.where(amax > 0, ex - 3, torch.full_like(ex, -127)).clamp(-127, 127)
        q = _round_e2m1(b * _pow2(-e).unsqueeze(-1))
        return q, (e + 127).to(torch.uint8), _pow2(e)
    s = (amax / (g * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    sv = s.float() * g
    r = torch.where(sv > 0, torch.ones_like(sv) / sv, torch.zeros_like(sv))
    return _round_e2m1(b * r.unsqueeze(-1)), s.view(torch.uint8), s.float()


def _pack(q):
    """Element values to codes, two to a byte (even column in the low half)."""
    a = q.abs()
    mag = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a * 0.5 + 4)).to(torch.uint8)
    code = (mag | (torch.signbit(q).to(torch.uint8) << 3)).view(q.shape[0], -1)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _tile_scales(s):
    """Scale bytes [rows, nblk] in tiles of 128 rows x 4 blocks: byte (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4."""
    rows, nb = s.shape
    rt, ct = -(-rows // 128), -(-nb // 4)
    p = torch.zeros((rt * 128, ct * 4), dtype=torch.uint8, device=s.device)
    p[:rows, :nb] = s
    return p.view(rt, 4, 32, ct, 4).permute(0, 3, 2, 1, 4).reshape(rt, ct, 512).contiguous()


def _untile_scales(t, rows, nb):
    rt, ct, _ = t.shape
    return t.view(rt, ct, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, ct * 4)[:rows, :nb]


def _decode(codes, scales, fmt):
    """fp32 values (without the tensor's scale) of packed codes and tiled scales."""
    rows = codes.shape[0]
    kp = codes.shape[1] * 2
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    lut = torch.cat([lut, -lut])
    c = torch.stack([codes & 15, codes >> 4], -1).view(rows, kp)
    s = _untile_scales(scales, rows, kp // BLOCK[fmt])
    sv = _pow2(s.int() - 127) if fmt == "mxfp4" else s.contiguous().view(torch.float8_e4m3fn).float()
    return (lut[c.int()].view(rows, -1, BLOCK[fmt]) * sv.unsqueeze(-1)).view(rows, kp)


def _weights(fmt, n, cols, gen):
    w = torch.randn((n, cols), generator=gen, device="cuda") * (1.0 / math.sqrt(cols))
    g = (w.abs().amax() / (448.0 * 6.0)).view(1) if fmt == "nvfp4" else None
    q, s, _ = _quantize(w, fmt, g)
    return _pack(q), _tile_scales(s), g


# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, rows, cols = case["op"], case["rows"], case["cols"]
    dt = DTYPES[case["dtype"]]
    st = dict(case)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    ru = lambda *s: torch.rand(s, generator=gen, device="cuda")  # noqa: E731
    ri = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, device="cuda")  # noqa: E731
    if op in ("quantize", "linear"):
        # activations with a few columns that are much larger, as hidden states have
        x = rn(rows, cols)
        x *= torch.where(ru(cols) < 0.01, 20.0, 1.0)
        st["x"] = x.to(dt)
        # a calibrated tensor scale: the largest magnitude expected over E4M3 x E2M1's largest
        st["gx"] = (90 + 20 * ru(1)) / (448 * 6) if case["fmt"] == "nvfp4" else None
    if op == "linear":
        st["w"], st["ws"], st["gw"] = _weights(case["fmt"], case["n"], cols, gen)
    if op == "product":
        st["a"], st["as"], st["ga"] = _weights(case["fmt"], rows, cols, gen)
        st["b"], st["bs"], st["gb"] = _weights(case["fmt"], case["n"], cols, gen)
    if op == "adjust":
        st["scores"] = (rn(rows, cols) * 3).to(dt)
        h = case["hist"]
        # token frequencies fall off: most of a history repeats few tokens
        st["history"] = (ru(rows, h) ** 4 * cols).to(torch.int32).clamp(max=cols - 1)
        st["history_len"] = ri(0, h + 1, rows).int()
        st["prompt_len"] = (st["history_len"].float() * ru(rows)).int()
        st["repetition"] = 1 + ru(rows) * 0.5
        st["presence"] = ru(rows)
        st["frequency"] = ru(rows) * 0.5
        st["temperature"] = 0.3 + ru(rows)
        nb = case["nb"]
        st["bias_ids"] = st["bias_vals"] = None
        if nb:
            ids = (torch.arange(nb, device="cuda") * (cols // nb) + ri(0, max(1, cols // nb), rows, nb)).int()
            st["bias_ids"] = torch.where(ru(rows, nb) < 0.2, torch.full_like(ids, -1), ids)
            st["bias_vals"] = rn(rows, nb) * 5
        st["mask"] = None
        if case["mask"] != "none":
            words = -(-cols // 32)
            mr = 1 if case["mask"] == "one" else rows
            m = ri(-2**31, 2**31, mr, words) & ri(-2**31, 2**31, mr, words)
            if mr > 2:
                m[1] = 0  # a row that its grammar leaves nothing
            st["mask"] = m.int()
    if op.startswith("distill"):
        t = rn(rows, cols) * 3
        st["scores"] = (t * 0.6 + rn(rows, cols) * 2).to(dt)
        # as kselect returns them for the negated teacher: ascending, ids beside them
        v, i = torch.topk(t, case["k"], dim=1)
        short = ru(rows, 1) < 0.1  # rows whose list ran short: (+inf, -1) at the tail
        tail = short & (torch.arange(case["k"], device="cuda") >= (case["k"] + 1) // 2)
        st["tv"] = torch.where(tail, torch.full_like(v, math.inf), -v).contiguous()
        st["ti"] = torch.where(tail, torch.full_like(i, -1), i).contiguous()
        scale = 4096.0 if case["dtype"] == "f16" else 1.0  # loss scaling, as half-precision training has
        st["row_grad"] = torch.where(ru(rows) < 0.05, 0.0, 1.0) * (scale / rows)
        if op == "distill_backward":
            st["stats"] = _stats(st["scores"].float(), case["temperature"])
    return st


# ---------------------------------------------------------------------------
# plain forms
def _stats(s, tau):
    m = s.amax(-1)
    return torch.stack([m, ((s - m.unsqueeze(-1)) / tau).exp().sum(-1)], -1)


def _teacher(st):
    t = -st["tv"]
    ok = (st["ti"] >= 0) & (t > -math.inf)
    z = torch.where(ok, t / st["temperature"], torch.full_like(t, -math.inf))
    z = z - z.amax(-1, keepdim=True)
    e = z.exp()
    tot = e.sum(-1, keepdim=True)
    return ok, e / tot, z - tot.log()


def _distill_loss(st, s, stats):
    tau = st["temperature"]
    ok, p, logp = _teacher(st)
    sl = s.gather(1, st["ti"].clamp(min=0))
    logq = (sl - stats[:, :1]) / tau - stats[:, 1:].log()
    return torch.where(ok, p * (logp - logq), torch.zeros_like(p)).sum(-1) * (tau * tau)


def _distill_grad(st, s, stats):
    tau = st["temperature"]
    ok, p, _ = _teacher(st)
    q = ((s - stats[:, :1]) / tau).exp() / stats[:, 1:]
    q.scatter_add_(1, st["ti"].clamp(min=0), torch.where(ok, -p, torch.zeros_like(p)))
    return (q * (st["row_grad"] * tau).unsqueeze(-1)).to(st["scores"].dtype)


def _adjust(st):
    x = st["scores"].float()
    rows, cols = x.shape
    hist, hl, pl = st["history"].long(), st["history_len"], st["prompt_len"]
    at = torch.arange(hist.shape[1], device=x.device)
    live = at < hl.unsqueeze(-1)
    after = live & (at >= pl.unsqueeze(-1))
    seen = torch.zeros_like(x).scatter_add_(1, hist, live.float())
    count = torch.zeros_like(x).scatter_add_(1, hist, after.float())
    col = lambda n: st[n].unsqueeze(-1)  # noqa: E731
    x = torch.where(seen > 0, torch.where(x > 0, x / col("repetition"), x * col("repetition")), x)
    x = x - count * col("frequency") - (count > 0).float() * col("presence")
    if st["bias_ids"] is not None:
        ids = st["bias_ids"].long()
        x = x.scatter_add(1, ids.clamp(min=0), torch.where(ids >= 0, st["bias_vals"], 0.0))
    x = x / col("temperature")
    if st["mask"] is not None:
        bit = torch.arange(32, device=x.device, dtype=torch.int32)
        allowed = ((st["mask"].unsqueeze(-1) >> bit) & 1).view(st["mask"].shape[0], -1)[:, :cols] != 0
        x = torch.where(allowed, x, -math.inf)
    return (-x if st["negate"] else x).to(st["scores"].dtype)


def _plain(st):
    op = st["op"]
    if op == "quantize":
        q, _, s = _quantize(st["x"], st["fmt"], st["gx"])
        v = q * s.unsqueeze(-1)
        if st["gx"] is not None:
            v = v * st["gx"]
        return {"values": v.view(st["rows"], -1)[:, :st["cols"]].to(st["x"].dtype)}
    if op == "product":
        y = _decode(st["a"], st["as"], st["fmt"]) @ _decode(st["b"], st["bs"], st["fmt"]).t()
        return {"out": y * (st["ga"] * st["gb"]) if st["ga"] is not None else y}
    if op == "linear":
        q, _, s = _quantize(st["x"], st["fmt"], st["gx"])
        v = (q * s.unsqueeze(-1)).view(st["rows"], -1)
        y = v @ _decode(st["w"], st["ws"], st["fmt"]).t()
        return {"out": (y * (st["gx"] * st["gw"]) if st["gx"] is not None else y).to(st["x"].dtype)}
    if op == "adjust":
        return {"out": _adjust(st)}
    s = st["scores"].float()
    if op == "distill_backward":
        return {"grad": _distill_grad(st, s, st["stats"])}
    stats = _stats(s, st["temperature"])
    loss = _distill_loss(st, s, stats)
    if op == "distill_forward":
        return {"loss": loss, "stats": stats}
    return {"loss": loss, "grad": _distill_grad(st, s, stats)}


def run(st):
    if not own:
        return _plain(st)
    B = _binding()
    op = st["op"]
    if op == "quantize":
        codes, scales = B.fp4_quantize(st["x"], st["fmt"], tensor_scale=st["gx"])
        return {"values": B.fp4_dequantize(codes, scales, st["cols"], st["fmt"],
                                           tensor_scale=st["gx"], dtype=st["x"].dtype)}
    if op == "product":
        return {"out": B.fp4_product(st["a"], st["as"], st["b"], st["bs"], st["fmt"],
                                     a_tensor_scale=st["ga"], b_tensor_scale=st["gb"])}
    if op == "linear":
        return {"out": B.fp4_linear(st["x"], st["w"], st["ws"], st["fmt"],
                                    x_tensor_scale=st["gx"], w_tensor_scale=st["gw"])}
    if op == "adjust":
        return {"out": B.score_adjust(st["scores"], history=st["history"],
                                      history_len=st["history_len"], prompt_len=st["prompt_len"],
                                      repetition=st["repetition"], presence=st["presence"],
                                      frequency=st["frequency"], bias_ids=st["bias_ids"],
                                      bias_vals=st["bias_vals"], temperature=st["temperature"],
                                      mask=st["mask"], negate=st["negate"])}
    tau = st["temperature"]
    if op == "distill_forward":
        loss, stats = B.topk_distill_forward(st["scores"], st["tv"], st["ti"], tau, negated=True)
        return {"loss": loss, "stats": stats}
    if op == "distill_backward":
        return {"grad": B.topk_distill_backward(st["scores"], st["tv"], st["ti"], st["stats"],
                                                st["row_grad"], tau, negated=True)}
    loss, grad = B.topk_distill(st["scores"], st["tv"], st["ti"], st["row_grad"], tau, negated=True)
    return {"loss": loss, "grad": grad}


# ---------------------------------------------------------------------------
def work(case):
    op, rows, cols = case["op"], case["rows"], case["cols"]
    sz = SIZE[case["dtype"]]
    if op in ("quantize", "product", "linear"):
        kp = -(-cols // 32) * 32
        packed = kp / 2 + kp / BLOCK[case["fmt"]]  # bytes of one packed row and its scales
    if op == "quantize":
        return {"bytes": rows * (2 * cols * sz + packed), "flops": 3 * rows * cols}
    if op == "product":
        return {"bytes": (rows + case["n"]) * packed + rows * case["n"] * sz,
                "flops": 2 * rows * case["n"] * cols}
    if op == "linear":
        return {"bytes": rows * cols * sz + case["n"] * packed + rows * case["n"] * sz,
                "flops": 2 * rows * case["n"] * cols}
    if op == "adjust":
        mask = {"none": 0, "one": cols / 8, "rows": rows * cols / 8}[case["mask"]]
        # half of each history is live on average
        return {"bytes": rows * (2 * cols * sz + case["hist"] * 2 + case["nb"] * 8 + 24) + mask,
                "flops": 4 * rows * cols}
    top = rows * case["k"] * 12 + rows * 12
    passes = {"distill_forward": 1, "distill_backward": 2, "distill": 2}[op]
    return {"bytes": rows * cols * sz * passes + top, "flops": 6 * rows * cols}


# ---------------------------------------------------------------------------
# the definitions in fp64
_GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _floor_log2(v):
    e = torch.floor(torch.log2(v.clamp(min=2.0 ** -200)))
    e = torch.where(torch.exp2(e + 1) <= v, e + 1, e)  # log2 itself may be an ulp off at a power of two
    return torch.where(torch.exp2(e) > v, e - 1, e)


def _exact_block_scale(amax, fmt, g):
    """Value of a block's scale (without g) from its largest magnitude, fp64."""
    if fmt == "mxfp4":
        return torch.exp2((_floor_log2(amax) - 2).clamp(-127, 127))
    v = (amax / (6 * g)).clamp(max=448.0)
    step = torch.exp2(_floor_log2(v.clamp(min=2.0 ** -6)) - 3)  # E4M3's spacing at v
    return torch.round(v / step) * step


def _exact_values(x, fmt, g):
    """x rounded to the format, without g, fp64 [rows, padded columns]."""
    rows, cols = x.shape
    blk = BLOCK[fmt]
    kp = -(-cols // 32) * 32
    b = torch.zeros((rows, kp), dtype=torch.float64, device=x.device)
    b[:, :cols] = x.double()
    b = b.view(rows, -1, blk)
    g = 1.0 if g is None else float(g)
    s = _exact_block_scale(b.abs().amax(-1), fmt, g)
    y = b / torch.where(s > 0, s * g, torch.full_like(s, math.inf)).unsqueeze(-1)
    a = y.abs()
    best = torch.zeros_like(a)
    for i in range(1, 8):  # past a midpoint the next value is nearer; a tie goes to the even code
        mid = (_GRID[i - 1] + _GRID[i]) / 2
        up = a >= mid if i % 2 == 0 else a > mid
        best = torch.where(up, torch.full_like(a, _GRID[i]), best)
    return (best * torch.sign(y) * s.unsqueeze(-1)).view(rows, kp)


def _exact_decode(codes, scales, fmt):
    rows, pitch = codes.shape
    grid = torch.tensor(_GRID + [-v for v in _GRID], dtype=torch.float64, device=codes.device)
    v = torch.empty((rows, pitch * 2), dtype=torch.float64, device=codes.device)
    v[:, 0::2] = grid[(codes % 16).long()]
    v[:, 1::2] = grid[torch.div(codes, 16, rounding_mode="floor").long()]
    r = torch.arange(rows, device=codes.device).unsqueeze(-1)
    c = torch.arange(pitch * 2 // BLOCK[fmt], device=codes.device).unsqueeze(0)
    s = scales[r // 128, c // 4, (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4].double()
    if fmt == "mxfp4":
        sv = torch.exp2(s - 127)
    else:
        ex, man = torch.div(s, 8, rounding_mode="floor"), s % 8
        sv = torch.where(ex > 0, (1 + man / 8) * torch.exp2(ex - 7), man / 8 * 2.0 ** -6)
    return v * sv.repeat_interleave(BLOCK[fmt], dim=1)


def _exact_adjusted(st, r):
    """Row r of the adjusted scores, fp64."""
    x = st["scores"][r].double()
    cols = x.numel()
    n, np_ = int(st["history_len"][r]), int(st["prompt_len"][r])
    toks = st["history"][r, :n].long()
    rep, pres, freq, temp = (float(st[v][r]) for v in ("repetition", "presence", "frequency", "temperature"))
    ids = torch.unique(toks)
    v = x[ids]
    x[ids] = torch.where(v > 0, v / rep, v * rep)
    cnt = torch.bincount(toks[np_:], minlength=cols)
    ids = torch.nonzero(cnt).view(-1)
    x[ids] -= freq * cnt[ids] + pres
    if st["bias_ids"] is not None:
        ok = st["bias_ids"][r] >= 0
        x[st["bias_ids"][r][ok].long()] += st["bias_vals"][r][ok].double()
    x /= temp
    if st["mask"] is not None:
        words = st["mask"][r if st["mask"].shape[0] > 1 else 0].long()
        c = torch.arange(cols, device=x.device)
        bits = torch.div(words[c // 32] % (1 << 32), 1 << (c % 32), rounding_mode="floor") % 2
        x[bits == 0] = -math.inf
    return -x if st["negate"] else x


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "quantize":
        v = _exact_values(st["x"], st["fmt"], st["gx"])[:, :st["cols"]]
        return {"values": v * st["gx"].double() if st["gx"] is not None else v}
    if op in ("product", "linear"):
        if op == "product":
            a, ga, b, gb = _exact_decode(st["a"], st["as"], st["fmt"]), st["ga"], st["b"], st["gb"]
            b = _exact_decode(b, st["bs"], st["fmt"])
        else:
            a, ga, gb = _exact_values(st["x"], st["fmt"], st["gx"]), st["gx"], st["gw"]
            b = _exact_decode(st["w"], st["ws"], st["fmt"])
        y = a @ b.t()
        return {"out": y * (ga.double() * gb.double()) if ga is not None else y}
    if op == "adjust":
        return {"out": torch.stack([_exact_adjusted(st, r) for r in range(st["rows"])])}
    tau, k = st["temperature"], st["k"]
    s = st["scores"].double() / tau
    loss = torch.zeros(st["rows"], dtype=torch.float64, device="cuda")
    lse = torch.logsumexp(s, 1)
    t = -st["tv"].double() / tau
    dead = st["ti"] < 0
    t = t.masked_fill(dead, -math.inf)
    p = torch.softmax(t, 1)
    ent = torch.where(p > 0, p * torch.log(p.clamp(min=1e-300)), torch.zeros_like(p)).sum(1)
    sl = torch.gather(s, 1, st["ti"].clamp(min=0))
    cross = (p * sl.masked_fill(dead, 0.0)).sum(1) - lse
    loss = (ent - cross) * tau * tau
    out = {}
    if op != "distill_backward":
        out["loss"] = loss
    if op == "distill_forward":
        m = st["scores"].double().amax(1)
        out["stats"] = torch.stack([m, torch.exp(lse - m / tau)], 1)
        return out
    grad = torch.exp(s - lse.unsqueeze(1))
    for j in range(k):  # one teacher entry of every row at a time
        grad.scatter_add_(1, st["ti"][:, j:j + 1].clamp(min=0), -p[:, j:j + 1])
    out["grad"] = grad * (st["row_grad"].double() * tau).unsqueeze(1)
    return out
