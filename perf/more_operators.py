"""Cases for the beam, embedding and adapter operators.

Each case is one call as a user of the library makes it:

* select    the best continuations of every request's beams, from score rows
* reorder   the beams' states (caches and histories) into the selected order
* lookup    rows of an embedding table, scaled
* gradient  the table's gradient, by token
* adapter   low-rank adapters of many requests added to a shared projection

The plain forms are elementary torch operations in fp32 (totals of beams in fp64: a
selection compares values that lie next to each other); `exact` restates the same
definitions in fp64.
"""

import math

import torch

own = False


DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
END = 2  # the token that a finished beam repeats


def _binding():
    from approximate_nearest_neighbour_gb300 import binding
    return binding


# ---------------------------------------------------------------------------
# cases
def listed():
    return [
        # one request, four beams, twice as many candidates: latency
        {"name": "select one request", "op": "select", "dtype": "f32", "groups": 1, "beams": 4,
         "cols": 32000, "k": 8, "masked": False},
        # an odd batch with a grammar's masked scores and odd rows
        {"name": "select masked", "op": "select", "dtype": "f16", "groups": 5, "beams": 5,
         "cols": 32001, "k": 10, "masked": True},
        # a serving batch over a large vocabulary
        {"name": "select batch", "op": "select", "dtype": "bf16", "groups": 64, "beams": 8,
         "cols": 131072, "k": 16, "masked": False},
        # one request's small caches and its history, after every token
        {"name": "reorder one request", "op": "reorder", "dtype": "bf16", "groups": 1, "beams": 4,
         "layers": 4, "heads": 8, "maxlen": 200, "dim": 128},
        # a batch's caches of two layers, filled to different lengths
        {"name": "reorder batch", "op": "reorder", "dtype": "bf16", "groups": 16, "beams": 4,
         "layers": 2, "heads": 8, "maxlen": 4096, "dim": 128},
        # the tokens that a decoding batch has just chosen
        {"name": "lookup 37 tokens", "op": "lookup", "dtype": "bf16", "tokens": 37,
         "rows": 32000, "cols": 4096},
        # a prompt batch's tokens from a large table
        {"name": "lookup prompt", "op": "lookup", "dtype": "bf16", "tokens": 8192,
         "rows": 131072, "cols": 4096},
        # a small evaluation batch over an odd number of vectors
        {"name": "gradient ragged", "op": "gradient", "dtype": "f32", "tokens": 777,
         "rows": 32001, "cols": 128},
        # a training step's tokens: the whole table's gradient
        {"name": "gradient step", "op": "gradient", "dtype": "bf16", "tokens": 16384,
         "rows": 32000, "cols": 4096},
        # one decoded token of one request
        {"name": "adapter one token", "op": "adapter", "dtype": "bf16", "tokens": 1, "cols": 4096,
         "n": 16384, "rank": 16, "adapters": 8, "runs": False},
        # a decoding batch of requests with adapters of their own
        {"name": "adapter 77 requests", "op": "adapter", "dtype": "bf16", "tokens": 77,
         "cols": 4096, "n": 16384, "rank": 16, "adapters": 64, "runs": False},
        # whole prompts of a few requests
        {"name": "adapter prompt", "op": "adapter", "dtype": "bf16", "tokens": 8192, "cols": 4096,
         "n": 16384, "rank": 64, "adapters": 6, "runs": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "reorder", "lookup", "gradient", "adapter"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "select":
        cols = _log(rng, 1000, 200_000)
        beams = rng.choice([1, 2, 3, 4, 5, 8, 10, 16])
        return {"op": op, "dtype": dtype, "groups": _log(rng, 1, max(1, min(128, 20_000_000 // (cols * beams)))),
                "beams": beams, "cols": cols, "k": _log(rng, 1, 48), "masked": rng.random() < 0.5}
    if op == "reorder":
        dim = rng.choice([64, 80, 128])
        heads, layers = rng.choice([1, 2, 8, 12]), rng.choice([1, 2, 3, 8])
        maxlen, beams = _log(rng, 10, 8192), rng.choice([2, 3, 4, 5, 8, 16])
        row = heads * layers * maxlen * dim * beams
        return {"op": op, "dtype": dtype, "groups": _log(rng, 1, max(1, min(64, 200_000_000 // row))),
                "beams": beams, "layers": layers, "heads": heads, "maxlen": maxlen, "dim": dim}
    if op in ("lookup", "gradient"):
        cols = _log(rng, 64, 8192)
        rows = _log(rng, 1000, min(200_000, 130_000_000 // cols))
        return {"op": op, "dtype": dtype, "tokens": _log(rng, 1, min(65536, 60_000_000 // cols)),
                "rows": rows, "cols": cols}
    cols, n = _log(rng, 256, 8192), _log(rng, 256, 16384)
    if rng.random() < 0.7:
        cols, n = -(-cols // 16) * 16, -(-n // 16) * 16
    rank = rng.choice([4, 8, 16, 24, 32, 64, 128])
    runs = rng.random() < 0.5
    tokens = _log(rng, 64, 8192) if runs else _log(rng, 1, 256)
    return {"op": op, "dtype": rng.choice(["f16", "bf16"]),
            "tokens": max(1, min(tokens, 100_000_000 // max(n, cols))), "cols": cols, "n": n,
            "rank": rank, "adapters": rng.choice([1, 3, 8]) if runs else _log(rng, 1, 64),
            "runs": runs}


# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    st = dict(case)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    ru = lambda *s: torch.rand(s, generator=gen, device="cuda")  # noqa: E731
    ri = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, device="cuda")  # noqa: E731
    if op == "select":
        g, b, cols = case["groups"], case["beams"], case["cols"]
        s = rn(g * b, cols) * 3
        if case["masked"]:
            s = torch.where(ru(g * b, cols) < 0.3, -math.inf, s)
        st["scores"] = s.to(dt)
        t = -(rn(g, b).abs() * 4).cumsum(1)
        # a request at its first token: only one beam is alive yet
        first = (ru(g, 1) < 0.1) & (torch.arange(b, device="cuda") > 0)
        st["totals"] = torch.where(first, -math.inf, t)
        st["finished"] = (ru(g, b) < 0.1) & ~first & (torch.arange(b, device="cuda") > 0)
    if op == "reorder":
        g, b = case["groups"], case["beams"]
        shape = (g * b, case["heads"], case["maxlen"], case["dim"])
        st["states"] = [rn(*shape).to(dt) for _ in range(case["layers"])]
        st["states"].append(ri(0, 32000, g * b, case["maxlen"]).int())
        st["axes"] = [2] * case["layers"] + [1]
        st["out"] = [torch.zeros_like(v) for v in st["states"]]
        # the better beams have more of the continuations
        st["beams_in"] = (ru(g, b) ** 2 * b).int().clamp(max=b - 1)
        st["lengths"] = ((0.25 + 0.75 * ru(g)) * case["maxlen"]).int().clamp(min=1)
    if op in ("lookup", "gradient"):
        t, rows, cols = case["tokens"], case["rows"], case["cols"]
        # token frequencies fall off; a few positions are padding and hold no token
        ids = (ru(t) ** 4 * rows).to(torch.int32).clamp(max=rows - 1)
        st["ids"] = torch.where(ru(t) < 0.02, -1, ids)
        st["scale"] = math.sqrt(cols)
        if op == "lookup":
            st["table"] = (rn(rows, cols) * 0.02).to(dt)
        else:
            st["grad"] = (rn(t, cols) * 0.01).to(dt)
    if op == "adapter":
        t, k, n, r, a = case["tokens"], case["cols"], case["n"], case["rank"], case["adapters"]
        st["x"] = rn(t, k).to(dt)
        st["a"] = (rn(a, r, k) / math.sqrt(k)).to(dt)
        st["b"] = (rn(a, n, r) * 0.1).to(dt)
        st["scales"] = (16.0 + 16.0 * ru(a)) / r
        st["base"] = rn(t, n).to(dt)
        if case["runs"]:  # tokens of one request follow each other; one request in seven has none
            start = (ru(t) < 4.0 / t).long()
            start[0] = 0
            kind = torch.where(ru(t) < 1 / 7, -1, ri(0, a, t))
            st["ids"] = kind[start.cumsum(0)].int()
        else:
            st["ids"] = torch.where(ru(t) < 0.1, -1, ri(0, a, t)).int()
            if t == 1:
                st["ids"] = ri(0, a, 1).int()
    return st


# ---------------------------------------------------------------------------
# plain forms
def _select(st):
    g, b, cols, k = st["groups"], st["beams"], st["cols"], st["k"]
    s = st["scores"].double()
    m = s.amax(-1, keepdim=True)
    lse = m + (s - m).exp().sum(-1, keepdim=True).log()
    total = (s - lse).view(g, b, cols) + st["totals"].double().unsqueeze(-1)
    only = torch.full_like(total, -math.inf)
    only[:, :, END] = st["totals"].double()
    total = torch.where(st["finished"].unsqueeze(-1), only, total).view(g, b * cols)
    at = torch.arange(b * cols, device=total.device)
    best, where = [], []
    for _ in range(k):  # the first of the largest, and on without it
        v = total.amax(1, keepdim=True)
        i = torch.where(total == v, at, b * cols).amin(1, keepdim=True)
        total.scatter_(1, i, -math.inf)
        best.append(v)
        where.append(i)
    v, i = torch.cat(best, 1), torch.cat(where, 1)
    ok = v > -math.inf
    return {"totals": v.float(), "beams": torch.where(ok, i // cols, -1).int(),
            "ids": torch.where(ok, i % cols, -1).int()}


def _reorder(st):
    g, b = st["beams_in"].shape
    src = (st["beams_in"].long() + torch.arange(g, device="cuda").unsqueeze(1) * b).view(-1)
    n = st["lengths"].repeat_interleave(b)
    for v, o, axis in zip(st["states"], st["out"], st["axes"]):
        shape = [1] * v.dim()
        shape[axis] = v.shape[axis]
        live = torch.arange(v.shape[axis], device="cuda").view(shape) < n.view([-1] + [1] * (v.dim() - 1))
        o.copy_(torch.where(live, v[src], o))
    return {str(i): o for i, o in enumerate(st["out"])}


def _plain(st):
    op = st["op"]
    if op == "select":
        return _select(st)
    if op == "reorder":
        return _reorder(st)
    if op == "lookup":
        ids = st["ids"].long()
        x = st["table"][ids.clamp(min=0)].float() * st["scale"]
        return {"out": torch.where((ids >= 0).unsqueeze(-1), x, 0.0).to(st["table"].dtype)}
    if op == "gradient":
        ids = st["ids"].long()
        g = st["grad"].float() * (ids >= 0).unsqueeze(-1)
        out = torch.zeros((st["rows"], st["cols"]), device="cuda")
        out.index_add_(0, ids.clamp(min=0), g)
        return {"grad": (out * st["scale"]).to(st["grad"].dtype)}
    a, r, k = st["a"].shape
    # every token through all adapters, all but its own masked out
    h = st["x"].float() @ st["a"].float().view(a * r, k).t()
    mine = st["ids"].unsqueeze(-1) == torch.arange(a, device="cuda")
    h = (h.view(-1, a, r) * (mine * st["scales"]).unsqueeze(-1)).view(-1, a * r)
    y = h @ st["b"].float().permute(0, 2, 1).reshape(a * r, -1)
    return {"out": (st["base"].float() + y).to(st["base"].dtype)}


def run(st):
    if not own:
        return _plain(st)
    B = _binding()
    op = st["op"]
    if op == "select":
        t, b, i = B.beam_select(st["scores"], st["totals"], st["k"], finished=st["finished"],
                                end_id=END)
        return {"totals": t, "beams": b, "ids": i}
    if op == "reorder":
        B.beam_reorder(st["states"], st["beams_in"], lengths=st["lengths"], axis=st["axes"],
                       out=st["out"])
        return {str(i): o for i, o in enumerate(st["out"])}
    if op == "lookup":
        return {"out": B.embedding_lookup(st["table"], st["ids"], st["scale"])}
    if op == "gradient":
        return {"grad": B.embedding_gradient(st["grad"], st["ids"], st["rows"], st["scale"])}
    return {"out": B.adapter_linear(st["x"], st["a"], st["b"], st["ids"], scales=st["scales"],
                                    base=st["base"])}


# ---------------------------------------------------------------------------
def work(case):
    op, sz = case["op"], SIZE[case["dtype"]]
    if op == "select":
        rows = case["groups"] * case["beams"]
        return {"bytes": rows * (case["cols"] * sz + 5) + case["groups"] * case["k"] * 12,
                "flops": 4 * rows * case["cols"]}
    if op == "reorder":
        g, b = case["groups"], case["beams"]
        # expected over the inputs' distribution: 5/8 of the positions are filled, and
        # beam s is taken by a continuation with probability sqrt((s + 1) / b) - sqrt(s / b)
        taken = sum(1 - (1 - (math.sqrt((s + 1) / b) - math.sqrt(s / b))) ** b for s in range(b))
        row = 0.625 * case["maxlen"] * (case["layers"] * case["heads"] * case["dim"] * sz + 4)
        return {"bytes": g * (taken + b) * row + g * (b + 1) * 4, "flops": 0}
    if op == "lookup":
        t, rows, cols = case["tokens"], case["rows"], case["cols"]
        # each row that is asked for is read once: row i is token's with probability p_i
        near = min(rows, 4096)
        hit = sum(1 - (1 - (((i + 1) / rows) ** 0.25 - (i / rows) ** 0.25)) ** t for i in range(near))
        lo, steps = near / rows, 2000
        for j in range(steps if near < rows else 0):  # the far rows by midpoints
            x = lo + (1 - lo) * (j + 0.5) / steps
            p = 0.25 * x ** -0.75 / rows
            hit += rows * (1 - lo) / steps * -math.expm1(t * math.log1p(-p))
        return {"bytes": (hit + t) * cols * sz + t * 4, "flops": t * cols}
    if op == "gradient":
        t, cols = case["tokens"], case["cols"]
        return {"bytes": (t + case["rows"]) * cols * sz + t * 4, "flops": 2 * t * cols}
    t, k, n, r = case["tokens"], case["cols"], case["n"], case["rank"]
    used = case["adapters"] * (1 - (1 - 1 / case["adapters"]) ** (4 if case["runs"] else t))
    return {"bytes": t * (k + 2 * n) * sz + used * r * (k + n) * sz + t * 4,
            "flops": 2 * t * r * (k + n)}


# ---------------------------------------------------------------------------
# the definitions in fp64
def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "select":
        g, b, cols, k = st["groups"], st["beams"], st["cols"], st["k"]
        tot, beam, tok = [], [], []
        for i in range(g):
            rows = st["scores"][i * b:(i + 1) * b].double()
            x = torch.log_softmax(rows, 1) + st["totals"][i].double().unsqueeze(1)
            done = st["finished"][i].nonzero().view(-1)
            x[done] = -math.inf
            x[done, END] = st["totals"][i, done].double()
            # of equal totals the lower beam, then the lower token, comes first
            v, at = torch.sort(x.view(-1), descending=True, stable=True)
            v, at = v[:k], at[:k]
            tot.append(v)
            beam.append(at.div(cols, rounding_mode="floor"))
            tok.append(at.remainder(cols))
        return {"totals": torch.stack(tot), "beams": torch.stack(beam).int(), "ids": torch.stack(tok).int()}
    if op == "reorder":
        out = {}
        for j, (v, axis) in enumerate(zip(st["states"], st["axes"])):
            o = torch.zeros(v.shape, dtype=torch.float64 if v.is_floating_point() else v.dtype, device=v.device)
            for r in range(v.shape[0]):
                i = r // st["beams"]
                s = i * st["beams"] + int(st["beams_in"][i, r % st["beams"]])
                n = int(st["lengths"][i])
                o[r].narrow(axis - 1, 0, n).copy_(v[s].narrow(axis - 1, 0, n))
            out[str(j)] = o
        return out
    ids = st["ids"].long()
    some = (ids >= 0).nonzero().view(-1)
    if op == "lookup":
        out = torch.zeros((st["tokens"], st["cols"]), dtype=torch.float64, device="cuda")
        out[some] = st["table"][ids[some]].double() * st["scale"]
        return {"out": out}
    if op == "gradient":
        out = torch.zeros((st["rows"], st["cols"]), dtype=torch.float64, device="cuda")
        out.index_put_((ids[some],), st["grad"][some].double(), accumulate=True)
        return {"grad": out * st["scale"]}
    out = st["base"].double()
    for i in range(st["adapters"]):
        t = (ids == i).nonzero().view(-1)
        h = st["x"][t].double() @ st["a"][i].double().t()
        out[t] += (h @ st["b"][i].double().t()) * st["scales"][i].double()
    return {"out": out}
