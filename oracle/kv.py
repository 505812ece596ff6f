"""The cache of keys and values in float64 (oracle; test infrastructure).

Plain loops over sequences and heads, written from the definitions:

* rope: pairs (x1, x2) turned by position * frequency radians, times a scale.
* slots: the i-th of n new tokens of a sequence of L is at position L - n + i, in the slot that the
  sequence's row of pages gives it.
* attend: out = sum_j p_j v_j, p the softmax of scale * q . k_j over the visible tokens of a sequence;
  zeros and a logarithm of -inf where a token sees nothing.
"""
from __future__ import annotations

import numpy as np


def rope(x, positions, freqs, layout="half", scale=1.0):
    """float64 [T, H, D]: the first 2 len(freqs) values of each head turned."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    d = 2 * len(freqs)
    for i, f in enumerate(np.asarray(freqs, np.float64)):
        a = np.asarray(positions, np.float64)[:, None] * f
        one, two = (i, i + d // 2) if layout == "half" else (2 * i, 2 * i + 1)
        y[..., one] = scale * (x[..., one] * np.cos(a) - x[..., two] * np.sin(a))
        y[..., two] = scale * (x[..., two] * np.cos(a) + x[..., one] * np.sin(a))
    return y


def slots(starts, lens, pages, page_size, T):
    """(slots, positions) int32 [T] of a well-formed batch."""
    s, p = np.full(T, -1, np.int32), np.zeros(T, np.int32)
    for b in range(len(lens)):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            at = lens[b] - n + i
            if at < 0:
                continue
            p[starts[b] + i] = at
            if at // page_size < len(pages[b]) and pages[b][at // page_size] >= 0:
                s[starts[b] + i] = pages[b][at // page_size] * page_size + at % page_size
    return s, p


def visible(n, L, causal=True, window=0, absent=()):
    """bool [n, L]: the i-th new token sees token j of the sequence."""
    at = np.arange(L - n, L)[:, None]
    j = np.arange(L)
    seen = np.ones((n, L), bool)
    if causal:
        seen &= j <= at
    if window:
        seen &= j > at - window
    seen[:, list(absent)] = False
    return seen


def attend(q, k, v, seen, scale):
    """q [n, H, D], k and v [L, Hk, D], seen [n, L], float64.  Returns (out [n, H, D], lse [n, H],
    mag [n, H, D] = sum_j p_j |v_j|, reach [n, H] = the largest scale * sum_d |q_d k_jd| in sight)."""
    n, H, D = q.shape
    G = H // k.shape[1] if k.shape[0] else H
    out, mag = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, reach = np.full((n, H), -np.inf), np.zeros((n, H))
    for i in range(n):
        js = np.nonzero(seen[i])[0]
        if not js.size:
            continue
        for h in range(H):
            kk, vv = k[js, h // G], v[js, h // G]
            s = scale * (kk @ q[i, h])
            top = s.max()
            e = np.exp(s - top)
            p = e / e.sum()
            out[i, h], mag[i, h] = p @ vv, p @ np.abs(vv)
            lse[i, h] = top + np.log(e.sum())
            reach[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, lse, mag, reach
