"""The mixture-of-experts operators in float64 (oracle; test infrastructure).

Plain loops over tokens and experts, written from the definitions:

* route: s = softmax(x) or sigmoid(x); choice = s + bias with a bias, the logits' own order
  without one; the best groups of experts stay (a group's best choice, or the sum of its two
  best); the k best choices, ties to the lowest index; weight = s, optionally over the sum,
  times a factor.  -inf logits (and -inf / NaN biases) are unavailable: id -1, weight 0 where
  nothing is left.  A row with a NaN or +inf: id -1, weight NaN everywhere.
* plan: assignments grouped by expert, in their own order within an expert.
* gemm: every expert's rows times its own weight, exactly dequantized operands.
* swiglu: silu(gate) * up, before any quantization.
* combine: add + sum_j w[t, j] * y[slot]; a slot of -1 contributes w * 0.
"""
from __future__ import annotations

import numpy as np

from .gemm import gemm_abs_ref, gemm_ref


def route(logits, k, *, score="softmax", bias=None, n_groups=1, top_groups=1, group_score="top2", renormalize=True,
          scale=1.0):
    """(ids int32 [T, k], weights float64 [T, k])."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    per = E // n_groups
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        row = x[t]
        if np.isnan(row).any() or (row == np.inf).any():
            weights[t] = np.nan
            continue
        free = row > -np.inf
        if not free.any():
            continue
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "softmax":
                e = np.exp(row - row[free].max())
                s = e / e.sum()
            else:
                s = 1.0 / (1.0 + np.exp(-row))
            choice = s if bias is None else s + np.asarray(bias, np.float64)
            key = row if bias is None else choice
            free = free & (key > -np.inf)
        groups = []
        for g in range(n_groups):
            mine = [e for e in range(g * per, (g + 1) * per) if free[e]]
            if group_score == "top2":
                val = sum(sorted((choice[e] for e in mine), reverse=True)[:2]) if mine else -np.inf
            else:
                val = max((key[e] for e in mine), default=-np.inf)
            groups.append((-val, g))
        kept = {g for _, g in sorted(groups)[:top_groups]}
        best = sorted((-key[e], e) for e in range(E) if free[e] and e // per in kept)[:k]
        pick = [e for _, e in best]
        w = s[pick]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        ids[t, :len(pick)], weights[t, :len(pick)] = pick, w * float(np.float32(scale))
    return ids, weights


def plan(ids, n_experts):
    """(offsets int32 [E + 1], order int32 [P], slots int32 [P])."""
    flat = np.asarray(ids).reshape(-1)
    order, slots, offsets = np.full(flat.size, -1, np.int32), np.full(flat.size, -1, np.int32), [0]
    for e in range(n_experts):
        mine = np.nonzero(flat == e)[0]
        at = np.arange(offsets[-1], offsets[-1] + mine.size)
        order[at], slots[mine] = mine, at
        offsets.append(offsets[-1] + mine.size)
    return np.array(offsets, np.int32), order, slots


def _rows(q, at):
    """The rows ``at`` of a quantized operand (fp8_row / fp8_block128)."""
    at = np.asarray(at)
    scales = q["scales"][at] if q["role"] == "activation" or q["scheme"] == "fp8_row" else \
        q["scales"][at[::128] // 128]
    return {**q, "rows": at.size, "codes": q["codes"][at], "scales": scales}


def gemm(a, w, offsets, order, top_k, gather):
    """(C, T): float64 [offsets[-1], N] products and sums of the products' magnitudes."""
    E = len(offsets) - 1
    N = w["rows"] // E
    C, T = np.zeros((offsets[-1], N)), np.zeros((offsets[-1], N))
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        at = np.arange(lo, hi)
        ae = _rows(a, np.asarray(order)[at] // top_k if gather else at)
        we = _rows(w, np.arange(e * N, (e + 1) * N))
        C[lo:hi], T[lo:hi] = gemm_ref(ae, we), gemm_abs_ref(ae, we)
    return C, T


def swiglu(x):
    """silu(gate) * up of float64 [rows, 2 F]."""
    F = x.shape[1] // 2
    g, u = np.asarray(x[:, :F], np.float64), np.asarray(x[:, F:], np.float64)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def combine(y, slots, weights, add=None):
    """(out, mag): float64 [T, N] sums and the sums of the terms' magnitudes."""
    w = np.asarray(weights, np.float64)
    T, k = w.shape
    out = np.zeros((T, y.shape[1])) if add is None else np.asarray(add, np.float64).copy()
    mag = np.abs(out)
    slots = np.asarray(slots).reshape(T, k)
    for t in range(T):
        for j in range(k):
            term = w[t, j] * (np.asarray(y[slots[t, j]], np.float64) if slots[t, j] >= 0 else np.zeros(y.shape[1]))
            out[t] += term
            mag[t] += np.abs(term)
    return out, mag
