"""GPU parity of the mixture-of-experts operators against the float64 oracle (oracle/moe.py).

Tolerances, derived before the first run:
* ids, offsets, order, slots: equal.
* routing weights: formed in fp32 or wider.  In fp32 the difference x - max is off by
  2^-24 |x - max|, the exponential by 2 ulp, a tree sum over at most 1024 experts by 22 roundings,
  quotient, renormalizing sum and factor by 8: (|x - max| + 32) 2^-24 relative.
* grouped products: tests/gemm_check.py's bounds (every element; bit for bit on exact operands).
* gated activation: h = g / (1 + 2^(-g log2 e)) u in fp32: the exponent's argument is off by
  2^-23 |g log2 e|, so the exponential by 2 |g| 2^-23 relative, the rest by 8 ulp, so h by
  (4 |g| + 16) 2^-24 =: eps |h|.  A scale is off by its maximum's eps and one rounding.  A code is
  the nearest e4m3 number to h / s, or the neighbour where h / s is within eps of the midpoint.
* combine: one rounding to bf16 (2^-8 relative) of an fp32 sum of k + 1 terms:
  2^-8 |out| + (k + 2) 2^-24 (sum of the terms' magnitudes).
"""
import numpy as np
import pytest
import torch

import oracle
import precision_quantized_linear_amd as pql
from gemm_check import check_gemm, check_gemm_exact, exact_operand, exact_precondition
from oracle import formats as F
from oracle import moe

pytestmark = pytest.mark.gpu

DEV = "cuda"
SENTINEL = 0x7FA5
INF = float("inf")


def up(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


def down(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# ---------------------------------------------------------------- route
def check_route(x, k, **kw):
    """``x``: a float tensor [T, E] on the device."""
    bias = kw.get("bias")
    ids, w = pql.moe_route(x, k, **kw)
    x64 = x.double().cpu().numpy()
    want_ids, want_w = moe.route(x64, k, **{**kw, "bias": None if bias is None else bias.cpu().numpy()})
    got_ids = ids.cpu().numpy()
    for t in np.nonzero((got_ids != want_ids).any(1))[0]:
        # Two groups' sums of two choices can be equal as numbers and not as sums of rounded
        # ones: {s1 + b, s2} and {s1, s2 + b}.  Which is kept is then up to the last bits, and
        # the row is checked against the oracle with the group scores that far apart taken as
        # the kernel took them; everywhere else ids are equal.
        assert kw.get("group_score") == "top2" and bias is not None
        want_ids[t], want_w[t] = _other_side_of_a_tie(x64[t], k, got_ids[t], kw, bias.cpu().numpy())
    assert np.array_equal(got_ids, want_ids)
    got = w.double().cpu().numpy()
    finite = np.where(np.isfinite(x64), x64, 0.0)
    spread = np.abs(finite).max(axis=1, keepdims=True) * 2
    nan = np.isnan(want_w)
    assert np.array_equal(np.isnan(got), nan)
    bad = np.abs(got - want_w) > (spread + 32) * 2.0 ** -24 * np.abs(want_w) + 2.0 ** -149
    assert not bad[~nan].any()


def _other_side_of_a_tie(row, k, got, kw, bias):
    """The oracle's route of one row with the kept groups chosen as ``got`` did where their sums
    tie.  A choice c = s + b is off by at most 4 ulp of max(|s|, |c|) <= 2 m (exponential,
    quotient, sum; m the largest |choice| or 1), a sum of two by twice that and one rounding, a
    difference of sums by twice that again: 40 m 2^-53."""
    E, n, top = row.size, kw["n_groups"], kw["top_groups"]
    per = E // n
    e = np.exp(row - row.max())
    s = e / e.sum() if kw["score"] == "softmax" else 1 / (1 + np.exp(-row))
    c = s + bias.astype(np.float64)
    score = np.sort(c.reshape(n, per), axis=1)[:, -2:].sum(1)
    tie = 40 * max(1.0, np.abs(c).max()) * 2.0 ** -53
    edge = np.sort(score)[::-1][top - 1]
    sure, open_ = score > edge + tie, np.abs(score - edge) <= tie
    used = np.zeros(n, bool)
    used[got // per] = True
    assert not (used & ~sure & ~open_).any()
    kept = sure | (open_ & used)
    assert kept.sum() <= top and kw.get("renormalize", True)
    ids = np.array([x for _, x in sorted((-c[x], x) for x in range(E) if kept[x // per])[:k]])
    return ids, s[ids] / s[ids].sum() * kw.get("scale", 1.0)


ROUTE_SHAPES = [(1, 1, 1), (1, 8, 8), (3, 5, 2), (17, 63, 7), (16, 64, 8), (33, 65, 6), (100, 128, 8), (257, 160, 6),
                (64, 256, 8), (9, 257, 1), (5, 512, 32), (7, 1000, 9), (2, 1024, 32)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,k", ROUTE_SHAPES)
def test_route_softmax(T, E, k, dtype):
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(E), dtype=torch.float32).to(DEV, dtype)
    check_route(x, k, renormalize=False)
    check_route(x, k, renormalize=True, scale=2.5)


@pytest.mark.parametrize("T,E,k", ROUTE_SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_bias(T, E, k, score):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, E, generator=g).to(DEV).bfloat16()       # many equal logits
    bias = (0.1 * torch.randn(E, generator=g)).to(DEV)
    check_route(x, k, score=score, bias=bias)
    check_route(x, k, score=score, bias=torch.zeros_like(bias), renormalize=False)   # ties of equal logits


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("E,n,top,k", [(64, 8, 4, 8), (256, 8, 4, 8), (160, 8, 3, 6), (60, 4, 1, 6), (12, 12, 5, 3),
                                       (1024, 64, 7, 32), (512, 2, 2, 4), (128, 64, 5, 10)])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("sigmoid", True), ("softmax", True)])
def test_route_groups(E, n, top, k, group_score, score, biased):
    g = torch.Generator().manual_seed(E + n)
    x = torch.randn(50, E, generator=g).to(DEV)
    bias = (0.05 * torch.randn(E, generator=g)).to(DEV) if biased else None
    check_route(x, k, score=score, bias=bias, n_groups=n, top_groups=top, group_score=group_score)


@pytest.mark.parametrize("E,n,top,k", [(64, 1, 1, 6), (100, 10, 3, 14), (256, 8, 4, 8), (250, 1, 1, 16), (512, 4, 2, 10),
                                       (96, 48, 20, 12)])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("sigmoid", True), ("softmax", True)])
def test_route_many_tokens(E, n, top, k, score, biased):
    """Several tokens per wave; the second half holds near ties: logits a few ulp apart, so that
    scores, and sums of two of them, agree to within fp32's rounding."""
    g = torch.Generator().manual_seed(E * k)
    x = torch.randn(2061, E, generator=g)
    close = 1.0 + torch.randint(-3, 4, (1030, E), generator=g).float() * 2.0 ** -23
    x[1031:] = torch.where(torch.rand(1030, E, generator=g) < 0.5, close, x[1031:])
    bias = (0.05 * torch.randint(-1, 2, (E,), generator=g).float()).to(DEV) if biased else None
    for group_score in ("max", "top2") if n > 1 else ("max",):
        check_route(x.to(DEV), k, score=score, bias=bias, n_groups=n, top_groups=top, group_score=group_score)


def test_route_ties_go_to_the_lowest_index():
    x = torch.zeros(5, 100, device=DEV)
    ids, w = pql.moe_route(x, 4)
    assert ids.tolist() == [[0, 1, 2, 3]] * 5 and torch.equal(w, torch.full_like(w, 0.25))
    check_route(x, 4, n_groups=10, top_groups=2, group_score="top2")
    check_route(x.bfloat16(), 7, score="sigmoid", bias=torch.zeros(100, device=DEV))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masked_and_broken_rows(score, biased, groups):
    x = torch.randn(9, 24, generator=torch.Generator().manual_seed(3))
    x[0] = -INF
    x[1, 1:] = -INF
    x[2, ::2] = -INF
    x[3, 5] = float("nan")
    x[4, 7] = INF
    x[5] = torch.finfo(torch.float32).min
    x[6, :12] = torch.finfo(torch.float32).min
    x[7] = 1000.0 * x[7]
    x[8, :20] = -INF
    bias = torch.randn(24, generator=torch.Generator().manual_seed(4)) if biased else None
    if biased:
        bias[2], bias[3], bias[9] = -INF, float("nan"), 50.0
    check_route(x.to(DEV), 6, score=score, bias=None if bias is None else bias.to(DEV), n_groups=groups,
                top_groups=max(1, groups - 1), group_score="top2")


@pytest.mark.parametrize("k", [0, -1, 9, 33, 1 << 40])
def test_route_refuses_a_k_outside_the_experts_before_any_allocation(k):
    logits = torch.zeros(4096, 8, device=DEV)
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(ValueError, match="k "):
        pql.moe_route(logits, k)
    assert torch.cuda.max_memory_allocated() - before < 1 << 30


def test_route_strided_rows_and_unaligned_start():
    buf = torch.randn(40, 131, device=DEV).bfloat16()
    check_route(buf[:, 3:67], 5)
    check_route(buf[::3, 1:129], 5, score="sigmoid")
    assert pql.moe_route(buf[:0, :64], 3)[0].shape == (0, 3)


# ---------------------------------------------------------------- plan
def check_plan(ids, E):
    p = pql.moe_plan(dev(ids.astype(np.int32)), E)
    offsets, order, slots = moe.plan(ids, E)
    assert np.array_equal(p.offsets.cpu().numpy(), offsets)
    assert np.array_equal(p.order.cpu().numpy(), order)
    assert np.array_equal(p.slots.cpu().numpy(), slots)
    return p


@pytest.mark.parametrize("T,k,E", [(0, 3, 5), (1, 1, 1), (1, 8, 64), (5, 3, 7), (24, 6, 160), (64, 8, 64), (171, 3, 65),
                                   (512, 1, 2), (513, 2, 1024), (1000, 8, 60), (4096, 8, 256), (9001, 7, 511),
                                   (30011, 8, 128), (70001, 8, 100)])
def test_plan(T, k, E):
    rng = np.random.default_rng(T + E)
    check_plan(rng.integers(0, E, (T, k)), E)
    check_plan(rng.integers(-2, E + 3, (T, k)), E)                       # some take no part
    check_plan((E * rng.random((T, k)) ** 4).astype(np.int64), E)        # crowded low experts


def test_plan_extremes():
    big = np.iinfo(np.int32)
    check_plan(np.full((300, 4), -1), 16)                                # nobody here
    check_plan(np.full((3000, 2), 15), 16)                               # everybody at the last expert
    check_plan(np.array([[big.min, big.max, 0, 16, 15, -1]] * 200), 16)


# ---------------------------------------------------------------- grouped products
def _ids(kind, T, k, E, seed):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full((T, k), E // 2)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k] if k <= E else rng.integers(0, E, (T, k))
    if kind == "dropped":
        ids = np.where(rng.random((T, k)) < 0.4, -1, ids)
    if kind == "crowded":
        ids = (E * rng.random((T, k)) ** 5).astype(np.int64)
    return ids


def _grouped(kind, T, k, E, seed):
    plan = pql.moe_plan(dev(_ids(kind, T, k, E, seed).astype(np.int32)), E)
    return plan, plan.offsets.cpu().numpy(), plan.order.cpu().numpy()


# one row, a few, tiles with tails, several tiles per expert; N past a tile and ragged, K of 1 .. 9 groups
GEMM_CASES = [
    ("fp8_block128", 1, 1, 1, 128, 128, "spread"), ("fp8_block128", 1, 8, 16, 256, 640, "spread"),
    ("fp8_block128", 37, 3, 10, 384, 384, "spread"), ("fp8_block128", 40, 2, 3, 512, 512, "dropped"),
    ("fp8_block128", 300, 2, 5, 384, 256, "crowded"), ("fp8_block128", 700, 1, 2, 640, 384, "spread"),
    ("fp8_block128", 290, 2, 4, 256, 128, "one"), ("fp8_block128", 1100, 3, 4, 768, 640, "spread"),
    ("fp8_row", 1, 1, 1, 8, 128, "spread"), ("fp8_row", 2, 6, 24, 130, 1152, "spread"),
    ("fp8_row", 37, 3, 10, 520, 384, "spread"), ("fp8_row", 40, 2, 3, 264, 512, "dropped"),
    ("fp8_row", 300, 2, 5, 33, 256, "crowded"), ("fp8_row", 700, 1, 2, 577, 384, "spread"),
    ("fp8_row", 290, 2, 4, 256, 128, "one"), ("fp8_row", 1100, 3, 4, 712, 512, "spread"),
    # tiles of 128 rows and columns past the last whole one
    ("fp8_block128", 300, 2, 5, 1408, 256, "crowded"), ("fp8_block128", 290, 2, 4, 1280, 128, "one"),
    ("fp8_row", 300, 2, 5, 1401, 256, "crowded"), ("fp8_row", 700, 1, 2, 1601, 384, "spread"),
    ("fp8_row", 500, 2, 4, 1032, 640, "dropped"),
    # passes of the stream split over workgroups, more of them than the mean asks for
    ("fp8_block128", 900, 1, 3, 128, 256, "crowded"), ("fp8_row", 1500, 2, 8, 100, 384, "one"),
    # the 256-row tiles: experts of a few rows to several tiles, columns past the last whole tile
    ("fp8_block128", 1430, 3, 130, 1024, 384, "spread"), ("fp8_block128", 1350, 2, 9, 8064, 256, "crowded"),
    ("fp8_row", 1430, 3, 130, 1000, 384, "dropped"), ("fp8_row", 1350, 2, 9, 8190, 256, "crowded"),
]


def test_gemm_cases_reach_every_kernel():
    names = {pql.moe_kernel_name(s, T, k, E, N, K, gather) for s, T, k, E, N, K, _ in GEMM_CASES for gather in (0, 1)}
    assert names == {f"k_moe_{n}, {s}>" for n in ("stream<1", "stream<4", "tile<128", "tile<256")
                     for s in ("fp8_row", "fp8_block128")}


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
def test_gemm_many_tiles_per_workgroup(scheme):
    """80 tiles of 256 x 256 per CU (the schedule's table holds 64): exact operands, so the fp32
    product of the decoded codes and power-of-two scales is exact and every element must equal its bf16
    rounding."""
    T, E, N, K = 20000, 2, 65536, 128
    plan, offsets, order = _grouped("spread", T, 1, E, 5)
    a, w = exact_operand(scheme, "activation", T, K, 3), exact_operand(scheme, "weight", E * N, K, 4)
    c = pql.moe_qgemm(pql.from_numpy(a, DEV), pql.from_numpy(w, DEV), plan, gather=True)
    table = dev(F.e4m3_decode(np.arange(256, dtype=np.uint8)).astype(np.float32))

    def decoded(q, repeat):
        s = dev(q["scales"]) if q["scales"].ndim == 1 else dev(q["scales"]).repeat_interleave(repeat, 0)
        return table[dev(q["codes"]).long()] * s.reshape(q["rows"], -1)

    A, W = decoded(a, 1), decoded(w, 128).view(E, N, K)
    for e in range(E):
        rows = plan.order[offsets[e]:offsets[e + 1]].long()
        for at in range(0, len(rows), 2048):
            want = (A[rows[at:at + 2048]] @ W[e].t()).bfloat16()
            got = c[int(offsets[e]) + at: int(offsets[e]) + at + want.shape[0]]
            assert torch.equal(got, want)


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("scheme,T,k,E,N,K,kind", GEMM_CASES)
def test_gemm_exact_every_element(scheme, T, k, E, N, K, kind, gather):
    plan, offsets, order = _grouped(kind, T, k, E, T + N)
    a = exact_operand(scheme, "activation", T if gather else T * k, K, 7 + T)
    w = exact_operand(scheme, "weight", E * N, K, 8 + N)
    exact_precondition(a, {**w, "rows": N, "codes": w["codes"][:N],
                           "scales": w["scales"][:N if scheme == "fp8_row" else N // 128]})
    out = torch.full((T * k + 3, N + 6), SENTINEL, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    inner = out[:T * k, 5:5 + N]                                        # unaligned rows
    pql.moe_qgemm(pql.from_numpy(a, DEV), pql.from_numpy(w, DEV), plan, gather=gather, out=inner)
    c64, _ = moe.gemm(a, w, offsets, order, k, gather)
    what = f"{pql.moe_kernel_name(scheme, T, k, E, N, K)} {scheme} T={T} k={k} E={E} N={N} K={K} {kind}"
    live = int(offsets[-1])
    check_gemm_exact(down(inner[:live]), c64, what)
    bits = down(out)
    bits[:live, 5:5 + N] = SENTINEL                                     # the rest as it was, tail rows included
    assert (bits == SENTINEL).all(), what
    aligned = pql.moe_qgemm(pql.from_numpy(a, DEV), pql.from_numpy(w, DEV), plan, gather=gather)
    assert np.array_equal(down(aligned[:live]), down(inner[:live])), what


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("scheme,T,k,E,N,K,kind", [
    ("fp8_block128", 3, 4, 8, 256, 2048, "spread"), ("fp8_block128", 150, 4, 6, 512, 1024, "crowded"),
    ("fp8_block128", 900, 2, 3, 384, 1920, "spread"), ("fp8_row", 3, 4, 8, 264, 2048, "spread"),
    ("fp8_row", 150, 4, 6, 512, 1024, "dropped"), ("fp8_row", 900, 2, 3, 392, 1920, "spread"),
])
def test_gemm_random(scheme, T, k, E, N, K, kind, gather):
    rng = np.random.default_rng(K)
    plan, offsets, order = _grouped(kind, T, k, E, K)
    x = F.f32_to_bf16_rne(rng.standard_normal((T if gather else T * k, K)).astype(np.float32))
    wt = F.f32_to_bf16_rne((0.02 * rng.standard_normal((E * N, K))).astype(np.float32))
    a, w = oracle.quantize(x, scheme, "activation"), oracle.quantize(wt, scheme, "weight")
    c = pql.moe_qgemm(pql.quantize(up(x), scheme), pql.quantize(up(wt), scheme, "weight"), plan, gather=gather)
    c64, mag = moe.gemm(a, w, offsets, order, k, gather)
    check_gemm(down(c[:int(offsets[-1])]), c64, mag, K, f"{scheme} T={T} {kind}")


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
@pytest.mark.parametrize("what,T,k,E,N,K,gather", [
    ("gathered activation", (1 << 20) + 5, 1, 2, 128, 4224, True), ("activation", (1 << 20) + 5, 1, 2, 128, 4224, False),
    ("result", (1 << 20) + 5, 1, 2, 4352, 128, False), ("weights", 300, 2, 130, 8192, 4352, True)])
def test_gemm_past_32_bit_offsets(scheme, what, T, k, E, N, K, gather):
    """Operands and results of more than 2^32 bytes: sampled rows, the first and last among them.

    The codes are uniform over all magnitudes, which check_gemm's accumulation term (8 K 2^-24 T) is
    not made for: the fp8 matrix instruction first sums groups of 8 products, cut at 2^-13 of the
    group's largest 2^(exponent of a + exponent of w) (measured: beside two cancelling 2^8 x 2^8,
    six products of 4 are lost, of 8 kept, of 12 count as 8).  The largest is exact, so a group
    loses at most 7 2^-13 of its largest product, all of them 7 2^-13 T: with
    T' = T (1 + 7 2^-13 / (8 K 2^-24)) = T (1 + 1792 / K) the term covers both."""
    g = torch.Generator(device=DEV).manual_seed(T + N)
    block = scheme == "fp8_block128"

    def operand(role, rows, scale_shape):
        codes = torch.randint(0, 127, (rows, K), dtype=torch.uint8, device=DEV, generator=g)   # no NaN codes
        if role == "weight":
            codes[:, ::3] += 128
        scales = torch.rand(scale_shape, device=DEV, generator=g) + 0.5
        return pql.QTensor(scheme, role, rows, K, codes, scales)

    rows = T if gather else T * k
    a = operand("activation", rows, (rows, K // 128) if block else (rows,))
    w = operand("weight", E * N, (E * N // 128, K // 128) if block else (E * N,))
    assert max(a.codes.numel(), w.codes.numel(), 2 * T * k * N) > 1 << 32
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device=DEV, generator=g)
    plan = pql.moe_plan(ids, E)
    c = pql.moe_qgemm(a, w, plan, gather=gather)
    table = dev(F.e4m3_decode(np.arange(256, dtype=np.uint8)).astype(np.float64))
    offsets, P = plan.offsets.cpu().numpy(), T * k
    at = np.unique(np.concatenate([[0, 1, P - 2, P - 1], np.random.default_rng(1).integers(0, P, 40),
                                   [x for o in offsets for x in (o - 1, o) if 0 <= x < P]]))
    for e in range(E):
        p = at[(at >= offsets[e]) & (at < offsets[e + 1])]
        if e % 16 and e != E - 1 and E > 16 or not len(p):
            continue
        p = torch.as_tensor(p, device=DEV)
        r = plan.order[p].long() // k if gather else p
        A = table[a.codes[r].long()] * (a.scales[r].double().repeat_interleave(128, 1) if block else a.scales[r].double()[:, None])
        ws = w.scales[e * (N // 128):(e + 1) * (N // 128)].double().repeat_interleave(128, 0).repeat_interleave(128, 1) \
            if block else w.scales[e * N:(e + 1) * N].double()[:, None]
        W = table[w.codes[e * N:(e + 1) * N].long()] * ws
        mag = (A.abs() @ W.abs().t()).cpu().numpy()
        check_gemm(down(c[p]), (A @ W.t()).cpu().numpy(), mag, K, f"{what} {scheme}", t_acc=mag * (1 + 1792 / K))


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
@pytest.mark.parametrize("T,E,N", [(40, 4, 256), (2000, 3, 512), (1300, 9, 8192)])
def test_gemm_keeps_a_broken_row_to_itself(scheme, T, E, N):
    """An infinite scale and NaN codes in one token's row, and in one expert's weight, change no
    other row: not the tile's neighbours, and not the tiles that follow in a workgroup."""
    K = 256
    plan, offsets, _ = _grouped("spread", T, 2, E, T)
    a = pql.quantize(torch.randn(T, K, device=DEV).bfloat16(), scheme)
    w = pql.quantize(torch.randn(E * N, K, device=DEV).bfloat16(), scheme, "weight")
    good = pql.moe_qgemm(a, w, plan, gather=True)
    rows = torch.zeros(2 * T, dtype=torch.bool, device=DEV)
    rows[plan.slots.view(T, 2)[17].long()] = True
    rows[int(offsets[1]):int(offsets[2])] = True           # expert 1
    a.scales.view(T, -1)[17] = INF
    a.codes[17, ::3] = 0x7F
    w.scales.view(E, -1)[1] = INF
    bad = pql.moe_qgemm(a, w, plan, gather=True)
    assert torch.equal(bad[~rows], good[~rows])
    assert not bad[rows].isfinite().any()


def test_gemm_follows_no_wild_plan():
    """Offsets and orders outside their ranges stay inside the buffers (and the call ends)."""
    plan, _, _ = _grouped("spread", 20, 2, 4, 1)
    a = pql.quantize(torch.randn(20, 256, device=DEV).bfloat16(), "fp8_row")
    w = pql.quantize(torch.randn(4 * 64, 256, device=DEV).bfloat16(), "fp8_row", "weight")
    plan.order[::3] = 1 << 30
    plan.order[1::3] = -7
    plan.offsets[:] = torch.tensor([-5, 1 << 30, 3, -(1 << 30), 50], dtype=torch.int32, device=DEV)
    out = torch.full((60, 64), SENTINEL, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    pql.moe_qgemm(a, w, plan, gather=True, out=out[:40])
    assert (down(out[40:]) == SENTINEL).all()
    plan.slots[:] = 1 << 30
    z = pql.moe_combine(torch.ones(40, 64, device=DEV).bfloat16(), plan, torch.ones(20, 2, device=DEV))
    assert not z.any()


# ---------------------------------------------------------------- gated activation
def _midpoint_ok(code, want, v, eps):
    a, b = F.e4m3_decode(code).astype(np.float64), F.e4m3_decode(want).astype(np.float64)
    steps = np.abs((code & 0x7F).astype(int) - (want & 0x7F).astype(int)) <= 1
    return (code == want) | (steps & (np.abs(v - (a + b) / 2) <= eps * np.abs(v)))


def check_swiglu(x, scheme, q):
    """``x``: bf16 bits [rows, 2 F]; q: the QTensor of the same rows."""
    x64 = F.bf16_to_f32(x).astype(np.float64)
    rows, cols = x64.shape[0], x64.shape[1] // 2
    h = moe.swiglu(x64)
    eps = (4 * np.abs(x64[:, :cols]) + 16) * 2.0 ** -24
    width = cols if scheme == "fp8_row" else 128
    top = np.abs(h).reshape(rows, -1, width)
    amax = top.max(2)
    slack = (np.abs(x64[:, :cols]).reshape(rows, -1, width).max(2) * 4 + 20) * 2.0 ** -24
    s = q.scales.double().cpu().numpy().reshape(rows, -1)
    want_s = np.where(amax > 0, amax / 448.0, 1.0)
    tiny = amax / 448.0 < 2.0 ** -120                       # near the subnormals and zero: checked as absolute
    assert (np.abs(s - want_s)[~tiny] <= (slack * want_s)[~tiny]).all()
    v = h / np.repeat(s, width, axis=1)
    code = q.codes.cpu().numpy()
    want = F.e4m3_encode(v)
    ok = _midpoint_ok(code, want, v, eps) | np.repeat(tiny, width, axis=1)
    assert ok.all(), f"{int((~ok).sum())} codes off, first at {tuple(np.argwhere(~ok)[0])}"


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
@pytest.mark.parametrize("M,F_", [(1, 128), (3, 256), (5, 1408), (130, 640), (9, 2048), (2, 2176), (3, 8192), (2, 9088),
                                  (1, 20480), (257, 128)])
def test_swiglu(scheme, M, F_):
    rng = np.random.default_rng(M * F_)
    x = F.f32_to_bf16_rne((2 * rng.standard_normal((M, 2 * F_))).astype(np.float32))
    check_swiglu(x, scheme, pql.swiglu_quantize(up(x), scheme))


def test_swiglu_row_of_odd_width():
    x = F.f32_to_bf16_rne(np.random.default_rng(5).standard_normal((7, 2 * 96)).astype(np.float32))
    check_swiglu(x, "fp8_row", pql.swiglu_quantize(up(x), "fp8_row"))


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
def test_swiglu_far_gates_zeros_and_strides(scheme):
    rng = np.random.default_rng(11)
    x = rng.standard_normal((12, 512)).astype(np.float32)
    x[0] = 0.0                                     # all zero: scale 1, codes 0
    x[1, :256] = -300.0                            # gates far below: the limit, 0
    x[2, :256] *= 60.0                             # exponentials that overflow
    x[3, 256:] = 0.0
    x[4] *= 1e-3
    x[5, :256] = 1e4
    wide = torch.full((12, 640), float("nan"), device=DEV).bfloat16()
    wide[:, 64:576] = torch.from_numpy(x).to(DEV).bfloat16()
    view = wide[:, 64:576]
    q = pql.swiglu_quantize(view, scheme)
    check_swiglu(down(view), scheme, q)
    assert (q.codes[0] & 0x7F == 0).all() and (q.scales.reshape(12, -1)[0] == 1).all()
    again = pql.swiglu_quantize(view, scheme, out=q)
    assert again is q
    check_swiglu(down(view), scheme, q)


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
def test_swiglu_leaves_rows_past_the_plan_alone(scheme):
    plan, offsets, _ = _grouped("dropped", 50, 3, 6, 9)
    live = int(offsets[-1])
    x = F.f32_to_bf16_rne(np.random.default_rng(3).standard_normal((150, 512)).astype(np.float32))
    q = pql._alloc_q(scheme, "activation", 150, 256, DEV)
    q.codes.fill_(0x7F)
    q.scales.fill_(-3.0)
    pql.swiglu_quantize(up(x), scheme, plan, out=q)
    head = pql.QTensor(scheme, "activation", live, 256, q.codes[:live], q.scales[:live])
    check_swiglu(x[:live], scheme, head)
    assert (q.codes[live:] == 0x7F).all() and (q.scales[live:] == -3.0).all()


# ---------------------------------------------------------------- combine
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 8, 4096), (5, 2, 24), (40, 6, 2056), (7, 3, 101), (130, 4, 640),
                                   (2, 32, 136), (300, 8, 2048)])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("kind", ["spread", "dropped"])
def test_combine(T, k, N, add, kind):
    rng = np.random.default_rng(T * N)
    plan, _, _ = _grouped(kind, T, k, 32, N)
    y = F.f32_to_bf16_rne(rng.standard_normal((T * k, N)).astype(np.float32))
    w = rng.random((T, k)).astype(np.float32)
    extra = F.f32_to_bf16_rne(rng.standard_normal((T, N)).astype(np.float32)) if add else None
    y64 = F.bf16_to_f32(y).astype(np.float64)
    want, mag = moe.combine(y64, plan.slots.cpu().numpy(), w,
                            None if extra is None else F.bf16_to_f32(extra).astype(np.float64))

    def check(out):
        got = F.bf16_to_f32(down(out)).astype(np.float64)
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (k + 2) * 2.0 ** -24 * mag).all()

    a_t = None if extra is None else up(extra)
    check(pql.moe_combine(up(y), plan, dev(w), add=a_t))
    wide = torch.full((T + 2, N + 9), SENTINEL, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    wide_y = torch.zeros(T * k, N + 5, device=DEV).bfloat16()
    wide_y[:, 3:3 + N] = up(y)
    check(pql.moe_combine(wide_y[:, 3:3 + N], plan, dev(w), add=a_t, out=wide[1:T + 1, 4:4 + N]))
    bits = down(wide)
    bits[1:T + 1, 4:4 + N] = SENTINEL
    assert (bits == SENTINEL).all()
    if add:                                                            # onto itself
        check(pql.moe_combine(up(y), plan, dev(w), add=a_t, out=a_t))


def test_broken_rows_of_logits_show_in_the_output():
    x = torch.randn(6, 8, device=DEV)
    x[2, 3] = float("nan")
    x[4] = -INF
    ids, w = pql.moe_route(x, 2)
    plan = pql.moe_plan(ids, 8)
    out = pql.moe_combine(torch.ones(12, 64, device=DEV).bfloat16(), plan, w)
    assert out[2].isnan().all() and not out[4].any()
    assert (out[[0, 1, 3, 5]].float() - 1).abs().max() <= 2.0 ** -8


# ---------------------------------------------------------------- together
def _layer(scheme, E, hidden, F_, seed):
    rng = np.random.default_rng(seed)
    w_in = F.f32_to_bf16_rne((0.05 * rng.standard_normal((E * 2 * F_, hidden))).astype(np.float32))
    w_out = F.f32_to_bf16_rne((0.05 * rng.standard_normal((E * hidden, F_))).astype(np.float32))
    return w_in, w_out, pql.quantize(up(w_in), scheme, "weight"), pql.quantize(up(w_out), scheme, "weight")


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
@pytest.mark.parametrize("T,k,E", [(1, 2, 4), (33, 3, 6), (260, 2, 3)])
def test_layer(scheme, T, k, E):
    """A whole layer against the oracle run on the device's own intermediate codes, step by step."""
    hidden, F_ = 256, 384
    rng = np.random.default_rng(T)
    w_in, w_out, qi, qo = _layer(scheme, E, hidden, F_, T)
    x = F.f32_to_bf16_rne(rng.standard_normal((T, hidden)).astype(np.float32))
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    ids, weights = pql.moe_route(logits, k)
    add = F.f32_to_bf16_rne(rng.standard_normal((T, hidden)).astype(np.float32))
    got = pql.moe_mlp(up(x), ids, weights, qi, qo, E, add=up(add))

    plan = pql.moe_plan(ids, E)
    offsets, order, slots = moe.plan(ids.cpu().numpy(), E)
    a, wi, wo = oracle.quantize(x, scheme, "activation"), oracle.quantize(w_in, scheme, "weight"), \
        oracle.quantize(w_out, scheme, "weight")
    h = pql.moe_qgemm(pql.quantize(up(x), scheme), qi, plan, gather=True)
    c64, mag = moe.gemm(a, wi, offsets, order, k, True)
    check_gemm(down(h), c64, mag, hidden, "first product")
    hq = pql.swiglu_quantize(h, scheme, plan)
    check_swiglu(down(h), scheme, hq)
    y = pql.moe_qgemm(hq, qo, plan)
    c64, mag = moe.gemm(pql.to_numpy(hq), wo, offsets, order, k, False)
    check_gemm(down(y), c64, mag, F_, "second product")
    want, mag = moe.combine(F.bf16_to_f32(down(y)).astype(np.float64), slots, weights.cpu().numpy(),
                            F.bf16_to_f32(add).astype(np.float64))
    out = F.bf16_to_f32(down(got)).astype(np.float64)
    assert (np.abs(out - want) <= 2.0 ** -8 * np.abs(want) + (k + 2) * 2.0 ** -24 * mag).all()


def test_layer_on_a_side_stream_and_captured():
    """The whole layer on another stream, then captured once and replayed on other inputs with
    eager work between the replays: every replay equals the eager result bit for bit."""
    scheme, T, k, E, hidden, F_ = "fp8_block128", 70, 2, 5, 256, 384
    _, _, qi, qo = _layer(scheme, E, hidden, F_, 1)
    x, logits = torch.empty(T, hidden, device=DEV).bfloat16(), torch.empty(T, E, device=DEV)

    def inputs(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x.copy_(torch.randn(T, hidden, device=DEV, generator=g))
        logits.copy_(torch.randn(T, E, device=DEV, generator=g) * seed)

    def layer():
        ids, weights = pql.moe_route(logits, k)
        return pql.moe_mlp(x, ids, weights, qi, qo, E)

    inputs(1)
    want = layer().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer()
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for seed in (2, 3, 4, 2):
        inputs(seed)
        want = layer().clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_empty_batch():
    ids = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    _, _, qi, qo = _layer("fp8_row", 2, 128, 128, 1)
    out = pql.moe_mlp(torch.empty(0, 128, device=DEV).bfloat16(), ids, torch.empty(0, 2, device=DEV), qi, qo, 2)
    assert out.shape == (0, 128)
