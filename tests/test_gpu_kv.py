"""GPU parity of rotary positions, slots, append, read and paged attention against the float64 oracle
(oracle/kv.py).  The attention's bounds: tests/kv_check.py.  Others, derived before the first run:

* slots, positions: equal.  Codes and scales of keys and values that are not turned: equal to the
  oracle's quantizer bit for bit; values read back: equal to its dequantization.
* rope: the angle in turns is exact to fp32's half step of half a turn, 2 pi 2^-26, sincospif to 2 ulp:
  cos and sin are off by less than 2^-21; two products and a sum in fp32 add 3 half steps of each
  product.  (|x1| + |x2|) |scale| 2^-20, and one rounding to bf16, 2^-8 |y|.
* turned keys: that without the rounding to bf16; a scale is off by its maximum's error, a code by
  half an e4m3 step of the exact value: 2^-4 |y| + 2^-10 s, and both errors again.
"""
import numpy as np
import pytest
import torch

import oracle
import precision_quantized_linear_amd as pql
from kv_check import DEV, SENTINEL, Filled, bf16_bits, check_attention, dev, expected, f64, run_case, up16
from oracle import formats as F
from oracle import kv as okv

pytestmark = pytest.mark.gpu


def down(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


# ---------------------------------------------------------------- rope
def check_rope(x64, got, positions, table, extra=0.0):
    freqs, d = table.freqs.cpu().numpy(), 2 * table.freqs.numel()
    want = okv.rope(x64, positions, freqs, table.layout, float(np.float32(table.scale)))
    other = np.abs(x64).copy()
    if table.layout == "half":
        other[..., : d // 2], other[..., d // 2: d] = other[..., d // 2: d].copy(), other[..., : d // 2].copy()
    else:
        other[..., 0:d:2], other[..., 1:d:2] = other[..., 1:d:2].copy(), other[..., 0:d:2].copy()
    tol = 2.0 ** -8 * np.abs(want) + (np.abs(x64) + other) * abs(table.scale) * 2.0 ** -20
    assert (np.abs(got - want) <= tol).all()
    assert np.array_equal(got[..., d:], x64[..., d:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,dim", [(1, 1, 16, 16), (1, 32, 128, 128), (3, 5, 64, 32), (7, 40, 128, 96),
                                       (130, 3, 192, 176), (33, 2, 256, 256), (5, 9, 80, 80), (2, 3, 72, 16),
                                       (700, 12, 128, 64)])
def test_rope(layout, T, H, D, dim):
    rng = np.random.default_rng(T * H + D + dim)
    bits = bf16_bits(rng.standard_normal((T, H, D)) * 3)
    pos = rng.integers(-1000, 1 << 20, T).astype(np.int32)
    pos[0] = 0 if T > 1 else (1 << 31) - 1
    table = pql.rope_freqs(dim, 10000.0, layout=layout, scaling={"type": "yarn", "factor": 8.0, "original": 4096},
                           device=DEV)
    x = up16(bits)
    got = pql.rope(x, dev(pos), table)
    assert np.array_equal(down(x), bits)
    check_rope(F.bf16_to_f32(bits).astype(np.float64), f64(got), pos, table)


def test_rope_in_place_in_a_projection():
    """Query and key heads of a [T, (H + 2 Hk) D] projection turned in place; values and the gap stay."""
    rng = np.random.default_rng(3)
    T, H, D = 37, 11, 128
    bits = bf16_bits(rng.standard_normal((T, (H + 2) * D + 8)))
    wide = up16(bits)
    pos = rng.integers(0, 5000, T).astype(np.int32)
    table = pql.rope_freqs(D, 500000.0, device=DEV)
    x = wide[:, : H * D].view(T, H, D)
    assert pql.rope(x, dev(pos), table, out=x).data_ptr() == wide.data_ptr()
    after = down(wide)
    assert np.array_equal(after[:, H * D:], bits[:, H * D:])
    check_rope(F.bf16_to_f32(bits[:, : H * D]).reshape(T, H, D).astype(np.float64),
               F.bf16_to_f32(after[:, : H * D]).reshape(T, H, D).astype(np.float64), pos, table)


def test_rope_head_major_out():
    """Heads outside, tokens inside, on both sides."""
    rng = np.random.default_rng(4)
    T, H, D = 19, 6, 64
    bits = bf16_bits(rng.standard_normal((H, T, D)))
    out = torch.full((H, T, D), 7.0, dtype=torch.bfloat16, device=DEV)
    pos = rng.integers(0, 100000, T).astype(np.int32)
    table = pql.rope_freqs(32, layout="interleaved", device=DEV)
    pql.rope(up16(bits).transpose(0, 1), dev(pos), table, out=out.transpose(0, 1))
    check_rope(F.bf16_to_f32(bits).transpose(1, 0, 2).astype(np.float64), f64(out).transpose(1, 0, 2), pos, table)


def test_rope_far_positions_keep_their_angle():
    """Neighbours 2^31 - 2 and 2^31 - 1 differ by one radian in the fastest pair."""
    table = pql.rope_freqs(16, device=DEV)
    x = torch.zeros((2, 1, 16), dtype=torch.bfloat16, device=DEV)
    x[:, :, 0] = 1.0
    pos = np.array([(1 << 31) - 2, (1 << 31) - 1], np.int32)
    got = f64(pql.rope(x, dev(pos), table))
    check_rope(f64(x), got, pos, table)


# ---------------------------------------------------------------- slots
@pytest.mark.parametrize("new,lens,ps,extra", [
    ([1], [1], 16, 0), ([1] * 24, list(range(1, 25)), 16, 0), ([0, 5, 0, 0, 3, 0], [7, 5, 0, 9, 40, 1], 16, 4),
    ([200, 1, 37], [200, 700, 38], 64, 3), ([3], [2], 16, 0), ([1] * 300, [100 + i for i in range(300)], 128, 1)])
def test_slots(new, lens, ps, extra):
    rng = np.random.default_rng(len(new))
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    width = max(lens) // ps + 2
    pages = rng.integers(0, 1000, (len(new), width)).astype(np.int32)
    pages[rng.random(pages.shape) < 0.05] = -1
    T = int(starts[-1]) + extra
    s, p = pql.kv_slots(dev(starts), dev(np.array(lens, np.int32)), dev(pages), ps, T)
    want_s, want_p = okv.slots(starts, lens, pages, ps, T)
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(p.cpu().numpy(), want_p)


def test_slots_past_the_pages_and_past_32_bits():
    starts, lens = dev(np.array([0, 3, 5], np.int32)), dev(np.array([18, 2], np.int32))
    pages = dev(np.array([[5], [1 << 27]], np.int32))
    s, p = pql.kv_slots(starts, lens, pages, 16, 5)
    assert s.tolist() == [5 * 16 + 15, -1, -1, -1, -1] and p.tolist()[:1] == [15]


def test_slots_of_no_sequences():
    s, p = pql.kv_slots(dev(np.zeros(1, np.int32)), dev(np.zeros(0, np.int32)), dev(np.zeros((0, 0), np.int32)), 16, 3)
    assert s.tolist() == [-1] * 3 and p.tolist() == [0] * 3


def test_slots_wild_batches_stay_inside():
    """Starts and lengths outside their ranges: an answer, slots of the pages or -1."""
    rng = np.random.default_rng(8)
    for seed in range(6):
        starts = rng.integers(-(1 << 31), 1 << 31, 9).astype(np.int32)
        lens = rng.integers(-(1 << 31), 1 << 31, 8).astype(np.int32)
        pages = rng.integers(-5, 50, (8, 4)).astype(np.int32)
        s, p = pql.kv_slots(dev(starts), dev(lens), dev(pages), 16, 77)
        s, p = s.cpu().numpy(), p.cpu().numpy()
        assert ((s >= -1) & (s < 50 * 16)).all() and (p >= 0).all()


# ---------------------------------------------------------------- append, read
def empty_cache(scheme, n_pages, ps, Hk, D, scales=(0.01, 0.02)):
    cache = pql.kv_cache(n_pages, ps, Hk, D, scheme, device=DEV,
                         **(dict(k_scale=scales[0], v_scale=scales[1]) if scheme == "fp8_tensor" else {}))
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x55)
    if scheme == "fp8_row":
        cache.k_scales.fill_(-7.0)
        cache.v_scales.fill_(-7.0)
    return cache


def stored(cache):
    return [None if t is None else t.view(torch.uint8).cpu().numpy().copy() if t.dtype != torch.float32
            else t.cpu().numpy().copy() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]


CACHES = [("fp8_row", 16, 1, 64), ("fp8_row", 64, 8, 128), ("fp8_row", 32, 3, 192), ("fp8_row", 16, 2, 256),
          ("fp8_tensor", 16, 5, 128), ("fp8_tensor", 128, 2, 192), ("bf16", 32, 4, 128), ("bf16", 16, 1, 256)]


@pytest.mark.parametrize("scheme,ps,Hk,D", CACHES)
@pytest.mark.parametrize("T", [1, 2, 37, 1500])
def test_append_and_read(scheme, ps, Hk, D, T):
    rng = np.random.default_rng(T + D + Hk)
    n_pages = -(-T // ps) + 2
    cache = empty_cache(scheme, n_pages, ps, Hk, D)
    before = stored(cache)
    slots = rng.permutation(n_pages * ps)[:T].astype(np.int32)
    slots[rng.random(T) < 0.2] = -1
    if T > 4:
        slots[3] = n_pages * ps              # one past the end: not written
    bits = []
    for spread in (1.0, 5.0):
        x = rng.standard_normal((T, Hk, D)) * np.exp(rng.uniform(-8, 3, (T, Hk, 1))) * spread
        x[rng.random((T, Hk)) < 0.1] = 0.0
        bits.append(bf16_bits(x))
    wide = torch.zeros((T, 2 * Hk * D + 8), dtype=torch.bfloat16, device=DEV)     # k and v in one projection
    k, v = wide[:, : Hk * D].view(T, Hk, D), wide[:, Hk * D: 2 * Hk * D].view(T, Hk, D)
    k.copy_(up16(bits[0]))
    v.copy_(up16(bits[1]))
    assert pql.kv_append(k, v, cache, dev(slots)) is cache
    live = (slots >= 0) & (slots < n_pages * ps)
    page, off = slots[live] // ps, slots[live] % ps
    after = stored(cache)
    got_k, got_v = pql.kv_read(cache, dev(slots))
    for i, got in enumerate((got_k, got_v)):
        want, values = before[i].copy(), np.zeros((T, Hk, D), np.uint16)
        if scheme == "bf16":
            w16 = want.view(np.uint16).reshape(n_pages, Hk, ps, D)
            w16[page, :, off] = bits[i][live]
            values[live] = bits[i][live]
        else:
            flat = bits[i].reshape(T * Hk, D)
            q = oracle.quantize(flat, "fp8_row") if scheme == "fp8_row" else \
                oracle.quantize_static(flat, "fp8_tensor", "activation", np.array([(0.01, 0.02)[i]], np.float32))
            want.reshape(n_pages, Hk, ps, D)[page, :, off] = q["codes"].reshape(T, Hk, D)[live]
            values[live] = oracle.dequantize(q).reshape(T, Hk, D)[live]
            if scheme == "fp8_row":
                ws = before[2 + i].copy()
                ws[page, :, off] = q["scales"].reshape(T, Hk)[live]
                assert np.array_equal(after[2 + i], ws)
        assert np.array_equal(after[i], want)
        assert np.array_equal(down(got), values)


@pytest.mark.parametrize("scheme,ps,Hk,D", CACHES)
@pytest.mark.parametrize("layout,part", [("half", 1.0), ("interleaved", 1.0), ("half", 0.5), ("interleaved", 0.25)])
def test_append_turned(scheme, ps, Hk, D, layout, part):
    rng = np.random.default_rng(D + Hk)
    T, n_pages = 70, 12 * 64 // ps
    cache = empty_cache(scheme, n_pages, ps, Hk, D)
    slots = rng.permutation(n_pages * ps)[:T].astype(np.int32)
    kb, vb = (bf16_bits(rng.standard_normal((T, Hk, D))) for _ in "kv")
    table = pql.rope_freqs(int(D * part), layout=layout, device=DEV)
    table.scale = 1.25
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    pql.kv_append(up16(kb), up16(vb), cache, dev(slots), table, dev(pos))
    want = okv.rope(F.bf16_to_f32(kb).astype(np.float64), pos, table.freqs.cpu().numpy(), layout, 1.25)
    page, off = slots // ps, slots % ps
    big = np.abs(want).max(-1, keepdims=True)
    eps = 2.0 ** -18 * big                                # (|x1| + |x2|) 1.25 2^-20 <= that, as |x1| + |x2| <= sqrt(2) big / 1.25 each way
    if scheme == "bf16":
        got = f64(cache.k)[page, :, off]
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + eps).all()
    else:
        codes = F.e4m3_decode(cache.k.cpu().numpy())[page, :, off]
        if scheme == "fp8_row":
            s = cache.k_scales.double().cpu().numpy()[page, :, off][..., None]
            assert (np.abs(s - big / 448) <= 2.0 ** -17 * big / 448).all()
        else:
            s = 0.01
            want = np.clip(want, -448 * s, 448 * s)
        assert (np.abs(codes * s - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * s + 2 * eps).all()
    plain = empty_cache(scheme, n_pages, ps, Hk, D)       # the values are as without a table
    pql.kv_append(up16(kb), up16(vb), plain, dev(slots))
    assert np.array_equal(stored(cache)[1], stored(plain)[1])


def test_append_broken_values_stay_visible():
    cache = empty_cache("fp8_row", 1, 16, 2, 64)
    x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device=DEV)
    x[0, 0, 5], x[1, 1, 7], x[2, 0] = float("nan"), float("inf"), 0.0
    pql.kv_append(x, x, cache, dev(np.array([0, 1, 2], np.int32)))
    k, _ = pql.kv_read(cache, dev(np.array([0, 1, 2], np.int32)))
    k = f64(k)
    assert np.isnan(k[0, 0, 5]) and np.isnan(k[0, 0]).sum() == 1 and np.isnan(k[1, 1, 7])
    assert (k[0, 1] == 1).all() and (k[1, 0] == 1).all() and (k[2, 0] == 0).all()
    static = empty_cache("fp8_tensor", 1, 16, 2, 64, scales=(1.0, 1.0))
    pql.kv_append(x * 1000, x, static, dev(np.array([0, 1, 2], np.int32)))
    k = f64(pql.kv_read(static, dev(np.array([0, 1, 2], np.int32)))[0])
    assert np.isnan(k[0, 0, 5]) and k[1, 1, 7] == 448 and (k[0, 1] == 448).all()


# ---------------------------------------------------------------- attention
SCHEMES = ["fp8_row", "fp8_tensor", "bf16"]


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("seqs", [[1], [17], [200, 1, 64, 33], [1000, 3]])
def test_one_token_each(scheme, D, seqs):
    run_case(D + len(seqs), scheme, seqs, [1] * len(seqs), 8, 2, D, 16)


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (16, 1), (20, 4), (7, 1), (40, 1), (12, 2), (128, 1)])
def test_head_layouts(scheme, H, Hk):
    run_case(H + Hk, scheme, [150, 47], [1, 3], H, Hk, 64, 32)
    run_case(H + Hk + 1, scheme, [150, 90], [40, 2], H, Hk, 128, 16)


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("new,seqs", [([5], [5]), ([100], [100]), ([64, 1, 130, 0, 33], [64, 500, 200, 77, 33]),
                                      ([257], [700]), ([2, 2, 2], [2, 65, 129]), ([20, 30], [700, 200]),
                                      ([40, 39], [1500, 40])])
def test_chunks(scheme, D, new, seqs):
    run_case(D + len(new), scheme, seqs, new, 4, 2, D, 16)


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 7, 64, 100, 5000])
def test_windows(scheme, causal, window):
    run_case(window, scheme, [300, 64, 90], [70, 64, 1], 4, 2, 128, 32, causal=causal, window=window)
    run_case(window, scheme, [900], [1], 4, 2, 64, 16, causal=causal, window=window)


@pytest.mark.parametrize("scheme", SCHEMES)
def test_not_causal(scheme):
    run_case(1, scheme, [130, 64, 1], [130, 3, 1], 4, 1, 64, 64, causal=False)


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 1024, 65536])
def test_page_sizes(scheme, ps):
    run_case(ps, scheme, [ps // 2 + 3, min(3 * ps, 2000) + 1, 100], [1, 20, 100], 4, 2, 64, ps)


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("new", [1, 3, 100])
def test_far_scores(scheme, new):
    """Logits of hundreds: almost all weight on one token; a scale below zero; a scale of zero."""
    run_case(2, scheme, [333], [new], 4, 2, 128, 16, spread=8.0, q_spread=8.0)
    run_case(3, scheme, [333], [new], 4, 2, 128, 16, scale=-0.5)
    run_case(4, scheme, [333], [new], 4, 2, 64, 16, scale=0.0)


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("new", [1, 40, 70])
def test_sees_nothing(scheme, new):
    """An empty sequence, more new tokens than the cache holds, sequences without pages: zeros and -inf."""
    fill, qb, got, lse = run_case(5, scheme, [0, 5, 200], [new, 9, new], 4, 2, 64, 16)
    assert (f64(got)[:new] == 0).all() and np.isneginf(f64(lse)[:new]).all()
    pages = torch.full_like(fill.pages, -1)
    got, lse = pql.kv_attention(up16(qb), fill.cache, fill.starts, fill.lens, pages, return_lse=True)
    assert (f64(got) == 0).all() and np.isneginf(f64(lse)).all()
    none = torch.empty((3, 0), dtype=torch.int32, device=DEV)
    got = pql.kv_attention(up16(qb), fill.cache, fill.starts, fill.lens, none)
    assert (f64(got) == 0).all()


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("new", [1, 25, 50])
@pytest.mark.parametrize("bad", [-1, 1 << 30, None])
def test_absent_pages(scheme, new, bad):
    """Tokens on a page outside the cache take no part."""
    rng = np.random.default_rng(6)
    fill = Filled(rng, scheme, [300, 90], 2, 64, 16, [new, new])
    qb = bf16_bits(rng.standard_normal((fill.T, 4, 64)))
    fill.pages[0, 3] = fill.n_pages if bad is None else bad
    fill.pages[0, 18] = -(1 << 31)
    got, lse = pql.kv_attention(up16(qb), fill.cache, fill.starts, fill.lens, fill.pages, return_lse=True)
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    gone = list(range(48, 64)) + list(range(288, 300))
    check_attention(fill, q64, f64(got), f64(lse), expected(fill, q64, absent={0: gone}))


@pytest.mark.parametrize("H,new", [(2, 1), (2, 6), (2, 50), (2, 100), (2, 200), (16, 3)])
@pytest.mark.parametrize("scheme,where", [(s, w) for s in SCHEMES for w in "kv"] + [("fp8_row", "scale")])
def test_a_broken_token_reaches_only_those_that_see_it(scheme, H, new, where):
    """A NaN (or, in scales and bf16, an infinity) stored for one token: rows before it are exact, rows
    from it on are NaN in the values it reaches."""
    rng = np.random.default_rng(7)
    L, D = 333, 128
    fill = Filled(rng, scheme, [L, 70], 2, D, 16, [new, 2])
    qb = bf16_bits(rng.standard_normal((fill.T, H, D)))
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    want = expected(fill, q64)
    j = L - 1 - new // 2
    page, off = int(fill.pages_np[0, j // 16]), j % 16
    for value in ([float("nan"), float("inf")] if scheme == "bf16" or where == "scale" else [float("nan")]):
        if where == "scale":
            fill.cache.v_scales[page, :, off] = value
        elif scheme == "bf16":
            (fill.cache.k if where == "k" else fill.cache.v)[page, :, off, 3] = value
        else:
            (fill.cache.k if where == "k" else fill.cache.v)[page, :, off, 3] = 0xFF
        got, lse = pql.kv_attention(up16(qb), fill.cache, fill.starts, fill.lens, fill.pages, return_lse=True)
        got, lse = f64(got), f64(lse)
        pos = np.arange(L - new, L)
        blind = np.concatenate([np.nonzero(pos < j)[0], [new, new + 1]])
        sees = np.nonzero(pos >= j)[0]
        check_attention(fill, q64, np.where(np.isnan(got), 1e30, got), lse, want, rows=blind)
        if where == "v":
            assert not np.isfinite(got[sees][..., 3]).any()
        elif value != value:
            assert np.isnan(got[sees]).all()


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("new", [1, 15, 30])
def test_rows_of_no_sequence_and_strides(scheme, new):
    """Rows before the first and behind the last sequence, columns beside the heads: left as they were.
    q and out are parts of wider rows, pages a part of a wider table."""
    rng = np.random.default_rng(8)
    fill = Filled(rng, scheme, [120, 70], 2, 128, 16, [new, new + 1])
    H, T = 10, fill.T + 7
    qb = bf16_bits(rng.standard_normal((T, H, 128)))
    wide_q = torch.full((T, H * 128 + 40), 3.0, dtype=torch.bfloat16, device=DEV)
    q = wide_q[:, 16: 16 + H * 128].view(T, H, 128)
    q.copy_(up16(qb))
    sentinel = up16(np.full((T, H + 1, 136), SENTINEL, np.uint16))
    out = sentinel[:, :H, :128]
    table = torch.full((2, fill.pages.shape[1] + 5), -9, dtype=torch.int32, device=DEV)
    table[:, : fill.pages.shape[1]] = fill.pages
    got = pql.kv_attention(q, fill.cache, fill.starts + 3, fill.lens, table[:, : fill.pages.shape[1]], out=out)
    assert got is out
    q64 = F.bf16_to_f32(qb[3: 3 + fill.T]).astype(np.float64)
    check_attention(fill, q64, f64(out)[3: 3 + fill.T], None, expected(fill, q64))
    left = down(sentinel)
    left[3: 3 + fill.T, :H, :128] = SENTINEL
    assert (left == SENTINEL).all()


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("new", [5, 30, 60])
def test_wild_batches_stay_inside(scheme, new):
    """Starts, lengths and pages outside their ranges: nothing outside out, no fault, rows of a sound
    sequence beside them exact."""
    rng = np.random.default_rng(9)
    fill = Filled(rng, scheme, [150] * 4, 2, 64, 16, [new] * 4)
    q = up16(bf16_bits(rng.standard_normal((fill.T, 4, 64))))
    for _ in range(8):
        starts = rng.integers(-(1 << 31), 1 << 31, 5).astype(np.int32)
        lens = rng.integers(-(1 << 31), 1 << 31, 4).astype(np.int32)
        pages = rng.integers(-(1 << 31), 1 << 31, fill.pages_np.shape).astype(np.int32)
        for s, l, p in ((starts, fill.lens, fill.pages), (fill.starts, lens, fill.pages), (fill.starts, fill.lens, pages),
                        (starts, lens, pages)):
            s, l, p = (x if isinstance(x, torch.Tensor) else dev(x) for x in (s, l, p))
            buf = up16(np.full((fill.T + 8, 4, 64), SENTINEL, np.uint16))
            pql.kv_attention(q, fill.cache, s, l, p, out=buf[4: 4 + fill.T])
            edge = down(buf)
            assert (edge[:4] == SENTINEL).all() and (edge[-4:] == SENTINEL).all()
    overlapping = dev(np.array([0, fill.T, 0, fill.T, 0], np.int32))      # every sequence claims every row
    pql.kv_attention(q, fill.cache, overlapping, fill.lens, fill.pages)
    torch.cuda.synchronize()


def test_empty_calls():
    cache = empty_cache("fp8_row", 1, 16, 2, 64)
    starts, lens = dev(np.zeros(3, np.int32)), dev(np.array([4, 0], np.int32))
    pages = dev(np.zeros((2, 1), np.int32))
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    i = torch.empty((0,), dtype=torch.int32, device=DEV)
    assert pql.kv_attention(e, cache, starts, lens, pages).shape == (0, 4, 64)
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    pql.kv_append(k, k, cache, i, pql.rope_freqs(64, device=DEV), i)
    assert pql.kv_read(cache, i)[0].shape == (0, 2, 64)
    assert pql.rope(e, i, pql.rope_freqs(64, device=DEV)).shape == (0, 4, 64)
    out = torch.full((2, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    none = torch.empty((0,), dtype=torch.int32, device=DEV)
    pql.kv_attention(out, cache, dev(np.zeros(1, np.int32)), none, pages[:0], out=out.clone())


def test_many_sequences():
    """More sequences than a wave has lanes, most of them without new tokens."""
    rng = np.random.default_rng(10)
    seqs = [int(x) for x in rng.integers(1, 60, 300)]
    new = [int(x) for x in rng.integers(0, 3, 300)]
    new[256] = 5
    seqs[256] = 500
    new = [min(a, b) for a, b in zip(new, seqs)]
    run = Filled(rng, "fp8_row", seqs, 1, 64, 16, new)
    qb = bf16_bits(rng.standard_normal((run.T, 2, 64)))
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    got, lse = pql.kv_attention(up16(qb), run.cache, run.starts, run.lens, run.pages, return_lse=True)
    check_attention(run, q64, f64(got), f64(lse), expected(run, q64))


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("new,seqs", [([1], [20000]), ([1] * 3, [9000, 5, 300]), ([2, 70], [6000, 3000]), ([15] * 2, [4000, 9000]),
                                      ([30] * 3, [4000, 200, 70])])
def test_long_contexts(scheme, new, seqs):
    run_case(12, scheme, seqs, new, 4, 1, 64, 64)


@pytest.mark.parametrize("scheme", ["fp8_row", "bf16"])
@pytest.mark.parametrize("new", [1, 20, 40])
@pytest.mark.parametrize("sizes", [(1e-6, 0.0), (1e-20, 0.0), (1e6, 1.0), (1e-8, 1.0), (1e30, 1e20), (1e-24, 1e-24)])
def test_value_sizes(scheme, new, sizes):
    """Tokens whose values are of very different sizes, rows of zeros (their scale is 1) among small ones, and a
    scale of exactly 1 that is none."""
    rng = np.random.default_rng(14)
    L, Hk, D = 300, 2, 128
    x = [rng.standard_normal((L, Hk, D)) for _ in "kv"]
    x[1] *= rng.choice(sizes, (L, Hk, 1))
    x[1][5] = 0.0
    x[1][L - new, :, 0], x[1][L - new, :, 1:] = 448.0 * (sizes[0] < 1e10), 0.0
    bits = [[bf16_bits(a) for a in x]]
    fill = Filled(rng, scheme, [L], Hk, D, 16, [new], bits=bits)
    qb = bf16_bits(rng.standard_normal((new, 4, D)) * 2)
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    got, lse = pql.kv_attention(up16(qb), fill.cache, fill.starts, fill.lens, fill.pages, return_lse=True)
    check_attention(fill, q64, f64(got), f64(lse), expected(fill, q64), small=L)


@pytest.mark.parametrize("scheme,n_pages", [("bf16", 80000), ("fp8_row", 150000), ("fp8_tensor", 150000)])
def test_past_32_bit_offsets(scheme, n_pages):
    """A cache of more than 2^32 bytes a half, its last pages in use: written, read, attended over by both kernels."""
    rng = np.random.default_rng(15)
    Hk, D, ps, L = 4, 128, 64, 200
    cache = pql.kv_cache(n_pages, ps, Hk, D, scheme, device=DEV,
                         **(dict(k_scale=0.01, v_scale=0.02) if scheme == "fp8_tensor" else {}))
    assert cache.k.numel() * cache.k.element_size() > 1 << 32
    pages = np.arange(n_pages - 4, n_pages, dtype=np.int32)[None, ::-1].copy()
    kb, vb = (bf16_bits(rng.standard_normal((L, Hk, D))) for _ in "kv")
    starts, lens = dev(np.array([0, L], np.int32)), dev(np.array([L], np.int32))
    slots, _ = pql.kv_slots(starts, lens, dev(pages), ps, L)
    pql.kv_append(up16(kb), up16(vb), cache, slots)
    small = Filled(rng, scheme, [L], Hk, D, ps, [L], bits=[[kb, vb]])
    k, v = pql.kv_read(cache, slots)
    ks, vs = pql.kv_read(small.cache, dev(okv.slots([0, L], [L], small.pages_np, ps, L)[0]))
    assert torch.equal(k, ks) and torch.equal(v, vs)
    for new in (L, 2):
        qb = bf16_bits(rng.standard_normal((new, 8, D)))
        starts = dev(np.array([0, new], np.int32))
        got = pql.kv_attention(up16(qb), cache, starts, lens, dev(pages))
        assert torch.equal(got, pql.kv_attention(up16(qb), small.cache, starts, lens, small.pages))


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("new", [1, 30, 60])
def test_a_workspace_of_the_callers_and_broken_queries(scheme, new):
    """Any bits in the workspace; a NaN or an infinity in one row of q reaches that row alone."""
    rng = np.random.default_rng(16)
    fill = Filled(rng, scheme, [3000, 1500], 2, 128, 16, [new, new])
    qb = bf16_bits(rng.standard_normal((fill.T, 4, 128)))
    q = up16(qb)
    need = pql.kv_attention_workspace(scheme, fill.T, 4, 2, 128, 2, fill.pages.shape[1], 16)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    want = pql.kv_attention(q, fill.cache, fill.starts, fill.lens, fill.pages)
    assert torch.equal(want, pql.kv_attention(q, fill.cache, fill.starts, fill.lens, fill.pages, workspace=ws))
    with pytest.raises(ValueError):
        pql.kv_attention(q, fill.cache, fill.starts, fill.lens, fill.pages, workspace=ws[:-1])
    q[new, 1, 7], q[0, 2, 9] = float("nan"), float("inf")
    got = pql.kv_attention(q, fill.cache, fill.starts, fill.lens, fill.pages, workspace=ws)
    assert torch.isnan(got[new, 1]).all() and torch.isnan(got[0, 2]).all()
    got[new, 1], got[0, 2] = want[new, 1], want[0, 2]
    assert torch.equal(got, want)


# ---------------------------------------------------------------- together
def layer(x, cache, batch, table, H, Hk, D):
    """One layer's attention from its projection x [T, (H + 2 Hk) D]."""
    starts, lens, pages = batch
    T = x.shape[0]
    slots, positions = pql.kv_slots(starts, lens, pages, cache.page_size, T)
    q = x[:, : H * D].view(T, H, D)
    k = x[:, H * D: (H + Hk) * D].view(T, Hk, D)
    v = x[:, (H + Hk) * D:].view(T, Hk, D)
    pql.kv_append(k, v, cache, slots, table, positions)
    return pql.kv_attention(pql.rope(q, positions, table), cache, starts, lens, pages)


@pytest.mark.parametrize("scheme", SCHEMES)
def test_layer_prompt_then_tokens(scheme):
    """A prompt in two chunks, then single tokens, against full attention over everything in float64 (from
    what the cache holds); another stream; and the last step captured and replayed with other inputs."""
    rng = np.random.default_rng(11)
    H, Hk, D, ps = 8, 2, 128, 16
    total = [90, 33]
    wide = (H + 2 * Hk) * D
    x = [bf16_bits(rng.standard_normal((n, wide))) for n in total]
    table = pql.rope_freqs(D, device=DEV)
    cache = empty_cache(scheme, 12, ps, Hk, D)
    pages = dev(rng.permutation(12)[:12].reshape(2, 6).astype(np.int32))
    steps = [[50, 20], [37, 10], [1, 1], [1, 1], [1, 1]]
    done = [0, 0]
    s = torch.cuda.Stream()
    for step, new in enumerate(steps):
        rows = np.concatenate([x[b][done[b]: done[b] + new[b]] for b in range(2)])
        done = [done[b] + new[b] for b in range(2)]
        batch = (dev(np.array([0, new[0], sum(new)], np.int32)), dev(np.array(done, np.int32)), pages)
        xin = up16(rows)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            y = layer(xin, cache, batch, table, H, Hk, D)
        torch.cuda.current_stream().wait_stream(s)
        slots, pos = pql.kv_slots(*batch, ps, sum(new))
        qr = f64(pql.rope(xin[:, : H * D].view(-1, H, D), pos, table))

        class Held:
            pass
        held = Held()
        held.D, held.scheme, held.new, held.seqs = D, scheme, new, list(done)
        held.starts_np = batch[0].cpu().numpy()
        held.k, held.v = [], []
        for b in range(2):
            at = np.arange(done[b])
            sl = pages.cpu().numpy()[b][at // ps] * ps + at % ps
            if scheme == "bf16":
                kv = [f64(t).transpose(0, 2, 1, 3).reshape(-1, Hk, D)[sl] for t in (cache.k, cache.v)]
            else:
                kv = [F.e4m3_decode(t.cpu().numpy()).transpose(0, 2, 1, 3).reshape(-1, Hk, D)[sl]
                      for t in (cache.k, cache.v)]
                for i, sc in enumerate((cache.k_scales, cache.v_scales)):
                    sc = f64(sc)
                    kv[i] = kv[i] * (sc if scheme == "fp8_tensor" else sc.transpose(0, 2, 1).reshape(-1, Hk)[sl][..., None])
            held.k.append(kv[0])
            held.v.append(kv[1])
        check_attention(held, qr, f64(y), None, expected(held, qr))
    # the next token, captured with fixed buffers, replayed with other rows and lengths
    xin = up16(x[0][:2])
    starts, lens = dev(np.array([0, 1, 2], np.int32)), dev(np.array([91, 34], np.int32))
    layer(xin, cache, (starts, lens, pages), table, H, Hk, D)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(xin, cache, (starts, lens, pages), table, H, Hk, D)
    for r in range(4):
        xin.copy_(up16(x[1][r: r + 2]))
        lens.copy_(dev(np.array([91 + r, 34 + (r % 2)], np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        got = down(y)
        assert np.array_equal(got, down(layer(xin, cache, (starts, lens, pages), table, H, Hk, D)))


def test_two_calls_at_once_and_the_same_every_time():
    """Two streams, a split context each: the same bits as one after the other, and on every run."""
    rng = np.random.default_rng(13)
    runs = [Filled(rng, sch, [3000, 700], 2, 128, 16, [1, 2]) for sch in ("fp8_row", "bf16")]
    qs = [up16(bf16_bits(rng.standard_normal((f.T, 8, 128)))) for f in runs]
    want = [down(pql.kv_attention(q, f.cache, f.starts, f.lens, f.pages)) for q, f in zip(qs, runs)]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for st, q, f in zip(streams, qs, runs):
            with torch.cuda.stream(st):
                got.append(pql.kv_attention(q, f.cache, f.starts, f.lens, f.pages))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert np.array_equal(down(g), w)
