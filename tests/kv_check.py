"""Caches, batches and the comparison with the float64 oracle for the tests of the cache of keys and
values.

Bounds, derived from the operations (u = 2^-24, fp32's half step):
* scores: a sum of D exact products in fp32, at most 8 D u of the products' magnitudes (the matrix
  cores' own order and cut, as for the GEMMs), scaled and taken to base 2 in three more roundings.  With
  reach = scale * sum_d |q_d k_jd| at its largest: delta = (8 D + 16) u reach.
* weights: exp2 of a difference of two such numbers, 2 ulp of its own: off by 2 delta + 2^-21 relative, as is
  their sum.  In 16 bits they are off by 2^-11 (fp16, beside 2^-25 of the largest weight's value, far
  below the rest) or 2^-8 (bf16).
* out: those errors on sum_j p_j |v_j| (mag), once for the weights and once for their sum, and one
  rounding to bf16, 2^-8 |out|.  The sums themselves are fp32: n_keys / 16 additions at most in a
  chain, below 2^-11 of mag up to 2^17 keys.
* small weights: under FP8 a weight is held in fp16 as 2^7 .. 2^15 times its share of the largest, so one
  below 2^-21 of it is off by up to 2^-32 of the largest, whose value reaches 448 somewhere in its row: with
  `small`, 2^-32 of the row's largest mag for each key.
* lse: delta, and 2^-22 of itself for the logarithm and the sum.
"""
import numpy as np
import torch

import oracle
import precision_quantized_linear_amd as pql
from oracle import formats as F
from oracle import kv as okv

DEV = "cuda"
SENTINEL = 0x7FA5


def up16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def f64(t):
    return t.double().cpu().numpy()


def bf16_bits(x):
    return F.f32_to_bf16_rne(np.asarray(x, np.float32))


class Filled:
    """A cache holding the given sequences' keys and values (bf16 bits [L, Hk, D] each), every other slot
    NaN (codes, scales and values), at random pages; with the batch's device tensors and the stored
    values in float64."""

    def __init__(self, rng, scheme, seqs, Hk, D, ps, new, *, spread=1.0, spare=3, bits=None, scales=(0.01, 0.02)):
        self.scheme, self.Hk, self.D, self.ps = scheme, Hk, D, ps
        need = [-(-L // ps) for L in seqs]
        self.n_pages = sum(need) + spare
        ids = rng.permutation(self.n_pages).astype(np.int32)
        width = max(need, default=0) + 1
        self.pages_np = np.full((len(seqs), width), -1, np.int32)
        shape = (self.n_pages, Hk, ps, D)
        codes = [np.full(shape, 0x7FFF if scheme == "bf16" else 0x7F, np.uint16 if scheme == "bf16" else np.uint8)
                 for _ in "kv"]
        row_scales = [np.full(shape[:3], np.nan, np.float32) for _ in "kv"]
        self.k, self.v = [], []
        at = 0
        for b, L in enumerate(seqs):
            mine = ids[at: at + need[b]]
            at += need[b]
            self.pages_np[b, : need[b]] = mine
            for i, stored in enumerate((self.k, self.v)):
                if bits is None:
                    x = rng.standard_normal((L, Hk, D)) * np.exp(rng.uniform(-1, 1, (L, Hk, 1))) * spread
                    xb = bf16_bits(x)
                else:
                    xb = bits[b][i]
                page, off = mine[np.arange(L) // ps], np.arange(L) % ps
                if scheme == "bf16":
                    codes[i][page, :, off] = xb
                    stored.append(F.bf16_to_f32(xb).astype(np.float64))
                elif L:
                    flat = xb.reshape(L * Hk, D)
                    q = oracle.quantize(flat, "fp8_row") if scheme == "fp8_row" else \
                        oracle.quantize_static(flat, "fp8_tensor", "activation", np.array([scales[i]], np.float32))
                    codes[i][page, :, off] = q["codes"].reshape(L, Hk, D)
                    if scheme == "fp8_row":
                        row_scales[i][page, :, off] = q["scales"].reshape(L, Hk)
                    stored.append(oracle.dequant_exact(q).reshape(L, Hk, D))
                else:
                    stored.append(np.zeros((0, Hk, D)))
        if scheme == "bf16":
            kv, s = [up16(c) for c in codes], [None, None]
        else:
            kv = [dev(c) for c in codes]
            s = [dev(r) for r in row_scales] if scheme == "fp8_row" else [dev(np.array([x], np.float32)) for x in scales]
        self.cache = pql.KVCache(scheme, self.n_pages, ps, Hk, D, *kv, *s)
        self.new = list(new)
        self.seqs = list(seqs)
        self.starts_np = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.starts = dev(self.starts_np)
        self.lens = dev(np.array(seqs, np.int32))
        self.pages = dev(self.pages_np)
        self.T = int(sum(new))


def expected(fill, q64, *, causal=True, window=0, scale=None, absent=None):
    """(out, lse, mag, reach) of the whole batch; ``absent``: {sequence: tokens that no page holds}."""
    scale = fill.D ** -0.5 if scale is None else scale
    parts = []
    for b, (n, L) in enumerate(zip(fill.new, fill.seqs)):
        lo = int(fill.starts_np[b])
        q = q64[lo: lo + n]
        lost = max(0, n - L)      # more new tokens than there are in the cache: the first see nothing
        seen = okv.visible(n, max(L, n), causal, window)[:, lost:] if lost else okv.visible(n, L, causal, window)
        if absent and b in absent:
            seen[:, list(absent[b])] = False
        parts.append(okv.attend(q, fill.k[b], fill.v[b], seen, float(np.float32(scale))))
    return [np.concatenate([p[i] for p in parts]) for i in range(4)]


def check_attention(fill, q64, got, got_lse, want, rows=None, small=0):
    out, lse, mag, reach = want
    rows = slice(None) if rows is None else rows
    delta = (8 * fill.D + 16) * 2.0 ** -24 * reach
    weight = 2.0 ** -8 if fill.scheme == "bf16" else 2.0 ** -11
    tol = 2.0 ** -8 * np.abs(out) + mag * (2 * (2 * delta + 2.0 ** -21) + 2 * weight + 2.0 ** -11)[..., None] + 2.0 ** -126
    tol = tol + small * 2.0 ** -32 * mag.max(-1, keepdims=True)
    err = np.abs(got - out)
    assert np.isfinite(got[rows]).all(), "not finite"
    worst = (err / tol)[rows].max() if got[rows].size else 0.0
    assert worst <= 1.0, f"error / bound = {worst:.3f}"
    if got_lse is not None:
        none = np.isneginf(lse)
        assert np.array_equal(np.isneginf(got_lse)[rows], none[rows])
        with np.errstate(invalid="ignore"):
            bad = ~none & ~(np.abs(got_lse - lse) <= delta + 2.0 ** -21 * (1 + np.abs(lse)))
        assert not bad[rows].any()


def run_case(seed, scheme, seqs, new, H, Hk, D, ps, *, causal=True, window=0, scale=None, spread=1.0, q_spread=1.0):
    rng = np.random.default_rng(seed)
    fill = Filled(rng, scheme, seqs, Hk, D, ps, new, spread=spread)
    qb = bf16_bits(rng.standard_normal((fill.T, H, D)) * q_spread)
    got, lse = pql.kv_attention(up16(qb), fill.cache, fill.starts, fill.lens, fill.pages, causal=causal, window=window,
                                scale=scale, return_lse=True)
    torch.cuda.synchronize()
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    check_attention(fill, q64, f64(got), f64(lse), expected(fill, q64, causal=causal, window=window, scale=scale))
    return fill, qb, got, lse
