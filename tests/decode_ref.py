"""Plain fp64 definitions of the beam, embedding and adapter calls, for their tests."""

import numpy as np


def log_softmax(row):
    """fp64 [cols], or None for a row without a softmax."""
    if np.isnan(row).any() or np.isposinf(row).any():
        return None
    m = row.max()
    if np.isneginf(m):
        return None
    d = row - m
    return d - np.log(np.exp(d).sum())


def continuations(scores, totals, finished=None, end_id=0):
    """Per group and beam, its continuations as (totals, ids), best first and the
    lower id of equal scores first."""
    groups, beams = totals.shape
    out = []
    for g in range(groups):
        lists = []
        for b in range(beams):
            t = float(totals[g, b])
            row = scores[g * beams + b]
            if not np.isfinite(t):
                lists.append((np.zeros(0), np.zeros(0, np.int64)))
            elif finished is not None and finished[g, b]:
                lists.append((np.array([t]), np.array([end_id])))
            else:
                lp = log_softmax(row)
                if lp is None:
                    lists.append((np.zeros(0), np.zeros(0, np.int64)))
                    continue
                order = np.argsort(-row, kind="stable")
                order = order[row[order] > -np.inf]
                lists.append((t + lp[order], order))
        out.append(lists)
    return out


def check_selection(got, scores, totals, k, finished=None, end_id=0):
    """A beam's share of a selection is the beginning of its own list, exactly; over
    beams the totals agree with the k largest up to the error of the fp32 sums of
    exponentials: cols / 256 + 64 additions in a row at most (a thread's chain and
    the joins), exponentials of 2 ulp whose arguments err by 2^-23 of themselves
    (x exp(-x) < 0.37), and the rounding of the result."""
    gt, gb, gi = (v.cpu().numpy() for v in got)
    groups, beams = totals.shape
    cols = scores.shape[1]
    for g, lists in enumerate(continuations(scores, totals, finished, end_id)):
        every = np.sort(np.concatenate([v for v, _ in lists]))[::-1][:k]
        n = len(every)
        assert (gb[g, n:] == -1).all() and (gi[g, n:] == -1).all() and np.isneginf(gt[g, n:]).all()
        e = (cols / 256 + 64) * 2.0 ** -24 + 2.0 ** -20
        tol = e + 2.0 ** -24 * 1.01 * np.abs(every)
        with np.errstate(over="ignore"):
            past = np.isinf(every.astype(np.float32))  # a total past fp32's range rounds to -inf
        assert np.isneginf(gt[g, :n][past]).all()
        tol[past] = np.inf
        got_t = np.where(past, every, gt[g, :n])
        assert (np.abs(got_t - every) <= tol).all(), (g, gt[g, :n], every)
        for b, (v, ids) in enumerate(lists):
            mine = gb[g, :n] == b
            m = int(mine.sum())
            assert np.array_equal(gi[g, :n][mine], ids[:m]), (g, b)
            assert (np.abs(got_t[mine] - v[:m]) <= tol[mine]).all()


def gradient(grad, ids, rows, scale, padding=-1):
    """(sums, sums of magnitudes, counts) per row, fp64."""
    out = np.zeros((rows, grad.shape[1]))
    mag = np.zeros_like(out)
    count = np.zeros(rows)
    for t, i in enumerate(ids):
        if 0 <= i < rows and i != padding:
            out[i] += grad[t]
            mag[i] += np.abs(grad[t])
            count[i] += 1
    return out * scale, mag * abs(scale), count


def adapter(x, a, b, ids, scales, base):
    """(result, what the second product's terms add up to in magnitude, the same of
    the first product carried through the second), fp64."""
    tokens, n = x.shape[0], b.shape[1]
    out = np.zeros((tokens, n)) if base is None else base.copy()
    second, first = np.zeros((tokens, n)), np.zeros((tokens, n))
    for t in range(tokens):
        i = int(ids[t])
        if 0 <= i < a.shape[0]:
            s = 1.0 if scales is None else float(scales[i])
            h = a[i] @ x[t]
            out[t] += s * (b[i] @ h)
            second[t] = abs(s) * (np.abs(b[i]) @ np.abs(h))
            first[t] = abs(s) * (np.abs(b[i]) @ (np.abs(a[i]) @ np.abs(x[t])))
    return out, second, first
