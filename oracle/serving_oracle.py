"""The serving calls restated in numpy fp64: packed prompts, the weight their
keys get, the paged cache and its eviction. Written from the formulas in
``include/rtp.h``, one sequence and head at a time; test infrastructure only.

Alongside each result stand the quantities that its error bounds need: the sum
of |p v| behind an output and the sum of |q k| behind a score.
"""
import numpy as np


def attended(n, window):
    """[n, n] truth values: row t attends key u."""
    t, u = np.arange(n)[:, None], np.arange(n)[None, :]
    return (u <= t) & (t - u < window)


def packed_head(q, k, v, window, scale):
    """One sequence and head (q, k, v fp64 [n, D]) -> o, lse, sum p|v|, scale * sum |q||k| (largest of a row)."""
    n = len(q)
    ok = attended(n, window)
    s = np.where(ok, scale * (q @ k.T), -np.inf)
    top = s.max(1, keepdims=True)
    e = np.exp(s - top)
    p = e / e.sum(1, keepdims=True)
    size = np.where(ok, scale * (np.abs(q) @ np.abs(k).T), 0.0)
    return p @ v, (top + np.log(e.sum(1, keepdims=True)))[:, 0], p @ np.abs(v), size.max(1)


def key_weights_head(q, k, lse, n_obs, window, scale):
    """One sequence and head -> the weight each key got from the last n_obs rows,
    that of the terms' |exponent| and the largest scale * sum |q||k| of a key."""
    n = len(q)
    ok = attended(n, window) & (np.arange(n)[:, None] >= n - n_obs)
    s = scale * (q @ k.T)
    e = np.where(ok, np.exp(np.where(ok, s - lse[:, None], 0.0)), 0.0)
    size = np.where(ok, scale * (np.abs(q) @ np.abs(k).T), 0.0)
    return e.sum(0), np.where(ok, np.abs(s) + np.abs(lse)[:, None], 0.0).max(0), size.max(0), ok.sum(0)


def decode_slots(n, window, sink):
    s = np.arange(n)
    return s[(s < sink) | (s >= n - window)]


def decode_head(q, k, v, slots, scale):
    """One query row over the rows `slots` of k, v [n, D] -> o, lse, p (per slot), sum p|v|, scale * sum |q||k|."""
    if len(slots) == 0:
        z = np.zeros(q.shape[0])
        return z, -np.inf, np.zeros(0), z, 0.0
    s = scale * (k[slots] @ q)
    e = np.exp(s - s.max())
    p = e / e.sum()
    return p @ v[slots], s.max() + np.log(e.sum()), p, p @ np.abs(v[slots]), scale * (np.abs(k[slots]) @ np.abs(q)).max()


def evict_slots(w, n, budget, sink, recent):
    """The slots kept of one sequence and KV head, from the weights w[:n]."""
    if n <= budget:
        return np.arange(n)
    slots = np.arange(n)
    fixed = (slots < sink) | (slots >= n - recent)
    rest = slots[~fixed]
    rank = np.where(np.isnan(w[rest]), np.inf, w[rest].astype(np.float64) + 0.0)
    first = np.isnan(w[rest]).astype(int)                     # NaN before every number
    order = np.lexsort((rest, -rank, -first))
    return np.sort(np.concatenate([slots[fixed], rest[order][:budget - fixed.sum()]]))


def append(pages, rows, cu, pos, table, page_size):
    """pages [P, page, ...] with the packed rows [T, ...] at their slots (a copy)."""
    out = pages.copy()
    for i in range(len(cu) - 1):
        for t in range(cu[i], cu[i + 1]):
            s = pos[i] + t - cu[i]
            if 0 <= s < table.shape[1] * page_size and 0 <= table[i, s // page_size] < len(pages):
                out[table[i, s // page_size], s % page_size] = rows[t]
    return out
