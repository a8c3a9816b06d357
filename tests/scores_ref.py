"""fp64 references of the 4-bit, score-adjustment and distillation entry points,
written from their definitions (numpy only)."""

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
MIDS = (E2M1[1:] + E2M1[:-1]) / 2
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def e4m3_values():
    """Values of the bytes 0 .. 126 (127 is NaN), ascending."""
    b = np.arange(127)
    ex, man = b >> 3, b & 7
    return np.where(ex > 0, (1 + man / 8) * 2.0 ** (ex - 7), man / 8 * 2.0 ** -6)


def e4m3_round(v):
    """Byte of the nearest E4M3 value, ties to the even byte, saturating."""
    vals = e4m3_values()
    hi = np.clip(np.searchsorted(vals, v), 1, 126)
    lo = hi - 1
    mid = (vals[lo] + vals[hi]) / 2
    up = (v > mid) | ((v == mid) & (hi % 2 == 0))
    return np.where(v >= vals[126], 126, np.where(up, hi, lo)).astype(np.uint8)


def scale_value(byte, fmt):
    byte = byte.astype(np.int64)
    if fmt == "mxfp4":
        return np.where(byte == 255, np.nan, 2.0 ** (byte - 127.0))
    return np.concatenate([e4m3_values(), [np.nan]])[byte]


def e2m1_round(y):
    """Code magnitude (0 .. 7) of |y|: nearest, ties to the even code, saturating."""
    a = np.abs(y)
    idx = np.zeros(a.shape, np.int64)
    for i in range(1, 8):
        idx = np.where((a >= MIDS[i - 1]) if i % 2 == 0 else (a > MIDS[i - 1]), i, idx)
    return idx


def blocks(x, fmt):
    rows, cols = x.shape
    kp = -(-cols // 32) * 32
    b = np.zeros((rows, kp))
    b[:, :cols] = x
    return b.reshape(rows, -1, BLOCK[fmt])


def block_scales(x, fmt, g=1.0):
    """Scale bytes [rows, nblk] from the definition in fp64."""
    b = blocks(x, fmt)
    with np.errstate(invalid="ignore"):
        amax = np.abs(b).max(-1)
        bad = ~np.isfinite(b).all(-1)
        if fmt == "mxfp4":
            _, e = np.frexp(amax)
            byte = np.where(amax > 0, np.clip(e - 1 - 2, -127, 127), -127) + 127
            return np.where(bad, 255, byte).astype(np.uint8)
        return np.where(bad, 127, e4m3_round(np.where(bad, 0, amax / (6 * g)))).astype(np.uint8)


def unpack(codes):
    """Signed element values [rows, 2 * pitch] of packed codes."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def untile(scales, rows, nblk):
    r = np.arange(rows)[:, None]
    c = np.arange(nblk)[None, :]
    return scales[r // 128, c // 4, (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4]


def values(codes, scales, fmt):
    """What packed rows stand for without the matrix's scale, fp64."""
    rows, pitch = codes.shape
    s = scale_value(untile(scales, rows, 2 * pitch // BLOCK[fmt]), fmt)
    return unpack(codes) * np.repeat(s, BLOCK[fmt], axis=1)


def adjust(x, history=None, history_len=None, prompt_len=None, repetition=None, presence=None,
           frequency=None, bias_ids=None, bias_vals=None, temperature=None, mask=None,
           negate=False):
    """(adjusted rows, bound on the sum of the magnitudes that went into each), fp64."""
    x = np.array(x, np.float64)
    mag = np.abs(x)
    rows, cols = x.shape
    for r in range(rows):
        if history is not None:
            n = history.shape[1] if history_len is None else int(history_len[r])
            n = max(0, min(n, history.shape[1]))
            p = 0 if prompt_len is None else max(0, min(int(prompt_len[r]), n))
            h = history[r, :n].astype(np.int64)
            ok = (h >= 0) & (h < cols)
            seen = np.unique(h[ok])
            rep = 1.0 if repetition is None else float(repetition[r])
            v = x[r, seen]
            with np.errstate(invalid="ignore"):
                x[r, seen] = np.where(v > 0, v / rep, v * rep)
            mag[r, seen] = np.abs(x[r, seen])
            out = h[p:][ok[p:]]
            cnt = np.bincount(out, minlength=cols)
            hit = np.nonzero(cnt)[0]
            pen = cnt[hit] * (0.0 if frequency is None else float(frequency[r]))
            pen = pen + (0.0 if presence is None else float(presence[r]))
            x[r, hit] -= pen
            mag[r, hit] += np.abs(pen)
        if bias_ids is not None:
            last = {}
            for i, c in enumerate(bias_ids[r]):
                if 0 <= c < cols:
                    last[int(c)] = float(bias_vals[r, i])
            for c, b in last.items():
                x[r, c] += b
                mag[r, c] += abs(b)
        if temperature is not None:
            x[r] /= float(temperature[r])
            mag[r] /= float(temperature[r])
        if mask is not None:
            m = mask[r if mask.shape[0] > 1 else 0].view(np.uint32)
            c = np.arange(cols)
            x[r, (m[c // 32] >> (c % 32).astype(np.uint32)) & 1 == 0] = -np.inf
    return (-x if negate else x), mag


def distill(s, tv, ti, tau, negated=False, row_grad=None):
    """(loss, m, Z, gradient, p dense) per row, fp64."""
    s = np.array(s, np.float64)
    rows, cols = s.shape
    loss, m, z = np.zeros(rows), np.zeros(rows), np.zeros(rows)
    grad, dense = np.zeros_like(s), np.zeros_like(s)
    for r in range(rows):
        m[r] = s[r].max()
        live = s[r] > -np.inf
        e = np.where(live, np.exp((np.where(live, s[r], 0) - (m[r] if live.any() else 0)) / tau), 0)
        z[r] = e.sum()
        q = e / z[r] if z[r] > 0 else e
        t = (-1.0 if negated else 1.0) * tv[r].astype(np.float64)
        ok = (ti[r] >= 0) & (ti[r] < cols) & (t > -np.inf)
        if not ok.any():
            continue
        w = np.exp((t[ok] - t[ok].max()) / tau)
        p = w / w.sum()
        logp = (t[ok] - t[ok].max()) / tau - np.log(w.sum())
        ids = ti[r][ok]
        with np.errstate(divide="ignore"):
            logq = np.where(s[r, ids] > -np.inf,
                            (np.where(live[ids], s[r, ids], 0) - (m[r] if live.any() else 0)) / tau,
                            -np.inf) - (np.log(z[r]) if z[r] > 0 else 0)
        loss[r] = tau * tau * np.sum(np.where(p > 0, p * (logp - logq), 0))
        np.add.at(dense[r], ids, p)
        if row_grad is not None and row_grad[r] != 0:
            grad[r] = row_grad[r] * tau * (q - dense[r])
    return loss, m, z, grad, dense
