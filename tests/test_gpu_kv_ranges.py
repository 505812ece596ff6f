"""Attention over contexts that are cut into ranges and joined, in each of its kernels (16, 32 and 128 rows per
tile), against the float64 oracle with the bounds of tests/kv_check.py.  Every case makes sure that the
kernel it means ran and that ranges were written to the workspace."""
import numpy as np
import pytest
import torch

import precision_quantized_linear_amd as pql
from kv_check import DEV, SENTINEL, Filled, bf16_bits, check_attention, dev, expected, f64, up16
from oracle import formats as F

pytestmark = pytest.mark.gpu

SCHEMES = ["fp8_row", "fp8_tensor", "bf16"]
KERNELS = {16: "k_attend_stream<16>+k_attend_join", 32: "k_attend_stream<32>+k_attend_join", 128: "k_attend_tile+k_attend_join"}
GUARD = 4096


def attend_cut(fill, q, rows, *, lens=None, pages=None, starts=None, out=None, cut=True, **kw):
    """One call in a workspace of exactly the bytes it asks for, whose surroundings stay as they were."""
    T, H, D = q.shape
    c, pages = fill.cache, fill.pages if pages is None else pages
    size = (c.scheme, T, H, c.n_kv_heads, D, pages.shape[0], pages.shape[1], c.page_size)
    assert pql.kv_kernel_name(*size) == KERNELS[rows]
    need = pql.kv_attention_workspace(*size)
    ws = torch.full((need + 2 * GUARD,), 0x77, dtype=torch.uint8, device=DEV)
    got = pql.kv_attention(q, c, fill.starts if starts is None else starts, fill.lens if lens is None else lens, pages,
                           out=out, workspace=ws[GUARD: GUARD + need], **kw)
    assert (ws[:GUARD] == 0x77).all() and (ws[GUARD + need:] == 0x77).all()
    assert not cut or (ws != 0x77).any(), "no context was cut"
    return got


def run_cut(seed, scheme, seqs, new, H, Hk, D, rows, ps=16, **kw):
    rng = np.random.default_rng(seed)
    fill = Filled(rng, scheme, seqs, Hk, D, ps, new)
    qb = bf16_bits(rng.standard_normal((fill.T, H, D)))
    got, lse = attend_cut(fill, up16(qb), rows, return_lse=True, **kw)
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    check_attention(fill, q64, f64(got), f64(lse), expected(fill, q64, **kw))


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 700, 1000, 1900])
@pytest.mark.parametrize("new,rows", [(5, 16), (30, 32), (60, 128)])
def test_windows_over_cut_contexts(scheme, causal, window, new, rows):
    """Windows that begin past key 0: ranges start there, and row tiles have fewer of them than their
    sequence's first; beside a sequence that is not cut."""
    run_cut(window + new, scheme, [2000, 300], [new, new], 4, 2, 128, rows, causal=causal, window=window)


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("windowed", [False, True])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("H,Hk,seqs,new,rows", [
    (2, 1, [900], 3, 16),                              # few joins: a workgroup per row
    (16, 16, [500, 470, 400, 511], 1, 16),             # many: four rows each
    (2, 1, [900, 700], 0, 32),
    (16, 16, [500, 430], 0, 32),
    (4, 2, [1500, 2500], 70, 128),
    (2, 2, [1537], 200, 128),
])
def test_every_join(scheme, D, H, Hk, seqs, new, rows, windowed):
    if rows == 32:     # the border lies at 32 rows to 128 values, at 64 above
        new = (33 if D <= 128 else 65) * Hk // H + (H > Hk)
    run_cut(D + H, scheme, seqs, [new] * len(seqs), H, Hk, D, rows, window=min(seqs) * 4 // 5 if windowed else 0)


CUT = [(2, 16), (25, 32), (70, 128)]


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("new,rows", CUT)
@pytest.mark.parametrize("bad", [-1, 1 << 30, None])
def test_absent_pages_of_cut_contexts(scheme, new, rows, bad):
    rng = np.random.default_rng(3)
    fill = Filled(rng, scheme, [1300, 90], 2, 64, 16, [new, new])
    qb = bf16_bits(rng.standard_normal((fill.T, 4, 64)))
    for p in (3, 40, 41, 42, 43, 44, 45, 46, 47, 70):
        fill.pages[0, p] = fill.n_pages if bad is None else bad
    gone = [j for j in range(1300) if j // 16 in (3, 40, 41, 42, 43, 44, 45, 46, 47, 70)]
    got, lse = attend_cut(fill, up16(qb), rows, return_lse=True)
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    check_attention(fill, q64, f64(got), f64(lse), expected(fill, q64, absent={0: gone}))


@pytest.mark.parametrize("new,rows", [(4, 16), (25, 16), (45, 32), (70, 128), (200, 128)])
@pytest.mark.parametrize("scheme,where", [(s, w) for s in SCHEMES for w in "kv"] + [("fp8_row", "scale")])
def test_a_broken_token_of_a_cut_context(scheme, new, rows, where):
    """A NaN or an infinity stored for one of the new tokens, or for one that the window hides from the later
    rows, reaches those that see it."""
    rng = np.random.default_rng(4)
    L, D, H = 1300, 128, 4
    fill = Filled(rng, scheme, [L, 70], 2, D, 16, [new, 2])
    qb = bf16_bits(rng.standard_normal((fill.T, H, D)))
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    pos = np.arange(L - new, L)
    for window, j in ((0, L - 1 - new // 2), (1100, L - new // 2 - 1100)):
        want = expected(fill, q64, window=window)
        sees = (pos >= j) & ((pos < j + window) if window else True)
        page, off = int(fill.pages_np[0, j // 16]), j % 16
        store = fill.cache.v_scales if where == "scale" else fill.cache.k if where == "k" else fill.cache.v
        at = (page, slice(None), off) if where == "scale" else (page, slice(None), off, 3)
        before = store[at].clone()
        for value in ([float("nan"), float("inf")] if scheme == "bf16" or where == "scale" else [0xFF]):
            store[at] = value
            got, lse = attend_cut(fill, up16(qb), rows, return_lse=True, window=window)
            got, lse = f64(got), f64(lse)
            blind = np.concatenate([np.nonzero(~sees)[0], [new, new + 1]])
            check_attention(fill, q64, np.where(np.isfinite(got), got, 1e30), lse, want, rows=blind)
            seeing = got[:new][sees]
            if where == "v":
                assert not np.isfinite(seeing[..., 3]).any()
            elif value != float("inf"):
                assert np.isnan(seeing).all()
        store[at] = before


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("new,rows", CUT)
def test_wild_neighbours_of_cut_contexts(scheme, new, rows):
    """Lengths and pages outside their ranges: the rows of the sequences that have sound ones are exact.  Wild starts
    besides: no byte outside the operands changes."""
    rng = np.random.default_rng(5)
    seqs = [1200, 1300, 1250, 1280]
    fill = Filled(rng, scheme, seqs, 2, 64, 16, [new] * 4)
    qb = bf16_bits(rng.standard_normal((fill.T, 4, 64)))
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    want = expected(fill, q64)

    def wild(shape):
        return rng.integers(-(1 << 31), 1 << 31, shape).astype(np.int32)

    def call(starts, lens, pages, **kw):
        buf = up16(np.full((fill.T + 8, 4, 64), SENTINEL, np.uint16))
        _, lse = attend_cut(fill, up16(qb), rows, starts=starts, lens=lens, pages=pages, out=buf[4: 4 + fill.T],
                            return_lse=True, **kw)
        edge = buf.view(torch.int16)
        assert (edge[:4] == SENTINEL).all() and (edge[-4:] == SENTINEL).all()
        return f64(buf[4: 4 + fill.T]), f64(lse)

    for step in range(6):
        lens, pages = np.array(seqs, np.int32), fill.pages_np.copy()
        bad = rng.permutation(4)[:2]
        if step % 3 != 1:
            lens[bad] = wild(2) if step < 3 else [(1 << 31) - 1, -1]
        if step % 3 != 0:
            pages[bad] = wild(pages[bad].shape)
        sound = np.concatenate([np.arange(b * new, (b + 1) * new) for b in range(4) if b not in bad])
        got, lse = call(fill.starts, dev(lens), dev(pages))
        check_attention(fill, q64, np.where(np.isfinite(got), got, 1e30), lse, want, rows=sound)
        call(dev(wild(5)), dev(lens), dev(pages), cut=False)
        call(dev(np.sort(wild(5))), dev(lens), dev(pages), cut=False)
    T = fill.T
    for starts in ([0, T, 0, T, 0], [T, 0, T, 0, T], [0, T, T, T, T], [-5, T, -7, T + 9, 3]):
        call(dev(np.array(starts, np.int32)), fill.lens, fill.pages, cut=False)


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("new,rows", CUT)
def test_cut_contexts_in_a_captured_call(scheme, new, rows):
    """Captured once, replayed over contexts of other lengths (some not cut at all) with eager calls between:
    the same bits as the eager call's, which the tests above hold to the oracle."""
    rng = np.random.default_rng(6)
    fill = Filled(rng, scheme, [2600, 700], 2, 64, 16, [new, new])
    q = torch.zeros((fill.T, 4, 64), dtype=torch.bfloat16, device=DEV)
    lens = fill.lens.clone()

    def call():
        return attend_cut(fill, q, rows, lens=lens, cut=False, return_lse=True)

    def eager_bits():
        return [t.view(torch.uint8).cpu() for t in call()]

    q.copy_(up16(bf16_bits(rng.standard_normal(q.shape))))
    eager_bits()
    size = (scheme, fill.T, 4, 2, 64, 2, fill.pages.shape[1], 16)
    ws = torch.empty((pql.kv_attention_workspace(*size),), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pql.kv_attention(q, fill.cache, fill.starts, lens, fill.pages, return_lse=True, workspace=ws)
    for step in ([2600, 700], [100, 90], [2599, 0], [1900, 650], [90, 700], [2600, 700]):
        lens.copy_(dev(np.array(step, np.int32)))
        q.copy_(up16(bf16_bits(rng.standard_normal(q.shape))))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.view(torch.uint8).cpu() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, eager_bits()))
