"""Attention over a paged key / value cache (oracle, test infrastructure only), in float64.

``visible`` lists what every query of one sequence sees; ``attend`` gives the outputs of one sequence together with
what a bound of their float32 computation needs; ``paged`` walks the sequences of a batch and their pages.

Pins (``tests/test_oracle_attention.py``): a pure-Python loop over single keys, equal keys giving the mean of the
values, one visible key giving its value, invariance under the order of pages, a chain tree being the causal
mask, and a window past the sequence being none.
"""

import numpy as np


def visible(n, l, window=0, sinks=0, mask=None, positions=None):
    """(n, l) truth values: which of its l keys each of a sequence's n queries (the last n keys' own) sees."""
    out = np.zeros((n, l), bool)
    for i in range(n):
        p = l - n + i
        if mask is not None and positions is not None:
            p = max(int(positions[i]), l - n)
        for j in range(l):
            node = j - (l - n)
            if mask is not None and node >= 0:
                out[i, j] = node < mask.shape[1] and bool(mask[i, node])
            elif mask is not None or j <= p:
                out[i, j] = window == 0 or j > p - window or j < sinks
    return out


def attend(q, k, v, seen, scale):
    """q (n, H, D), k and v (l, Hk, D), seen (n, l) -> (out, absolute, spread, total), float64: the outputs; sum_j P_j |v_j|;
    the largest sum_d |q_d k_jd| scale of a row; and sum_j exp(score_j - largest) with sum_j |v_j| over it."""
    n, H, D = q.shape
    l, Hk, _ = k.shape
    out = np.zeros((n, H, D))
    absolute = np.zeros((n, H, D))
    small = np.zeros((n, H, D))
    spread = np.zeros((n, H))
    for h in range(H):
        kh, vh = k[:, h * Hk // H].astype(np.float64), v[:, h * Hk // H].astype(np.float64)
        qh = q[:, h].astype(np.float64)
        for i in range(n):
            at = seen[i]
            if not at.any():
                continue
            s = (kh[at] @ qh[i]) * scale
            w = np.exp(s - s.max())
            out[i, h] = (w / w.sum()) @ vh[at]
            absolute[i, h] = (w / w.sum()) @ np.abs(vh[at])
            small[i, h] = np.abs(vh[at]).sum(0) / w.sum()
            spread[i, h] = (np.abs(kh[at]) @ np.abs(qh[i])).max() * scale
    return out, absolute, spread, small


def paged(q, k_cache, v_cache, table, lens, starts, scale, window=0, sinks=0, mask=None, positions=None):
    """q (T, H, D), caches (pages, page_size, Hk, D): ``attend`` of every sequence, rows of no sequence NaN; keys on pages
    that are not in the pool are not seen."""
    T, H, D = q.shape
    pages, size, Hk, _ = k_cache.shape
    res = [np.full((T, H, D), np.nan), np.zeros((T, H, D)), np.zeros((T, H)), np.zeros((T, H, D))]
    for b in range(len(lens)):
        l = min(max(int(lens[b]), 0), table.shape[1] * size)
        r0, n = int(starts[b]), int(starts[b + 1] - starts[b])
        rows = slice(r0, r0 + n)
        seen = visible(n, l, window, sinks, None if mask is None else mask[rows],
                       None if positions is None else positions[rows])
        page = table[b, np.arange(l) // size].astype(np.int64)
        ok = (page >= 0) & (page < pages)
        seen &= ok[None, :]
        used = seen.any(0)
        k, v = np.zeros((l, Hk, D)), np.zeros((l, Hk, D))
        at = np.flatnonzero(used)
        k[at] = k_cache[page[at], at % size]
        v[at] = v_cache[page[at], at % size]
        for to, x in zip(res, attend(q[rows], k, v, seen, scale)):
            to[rows] = x
    return res
