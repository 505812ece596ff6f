"""Edges of the mixture-of-experts operators on the GPU, against the float64 oracle (oracle/moe.py)."""
import numpy as np
import pytest
import torch

import precision_quantized_linear_amd as pql
from gemm_check import check_gemm_exact, exact_operand
from oracle import formats as F
from oracle import moe
from test_gpu_moe import down, up

pytestmark = pytest.mark.gpu

DEV = "cuda"


# ---------------------------------------------------------------- gated activation
def check_swiglu_everywhere(x, scheme, q):
    """Every scale and code of bf16 bits ``x`` [rows, 2 F], whatever their size.

    h is off by eps |h|, eps = (4 |g| + 16) 2^-24 (the exponent's argument is off by 2^-23 |g log2 e|,
    the rest by less than 8 ulp), and by 2^-150 where it is subnormal (half a step of that grid).  A
    scale is the rounded quotient of the largest |h| and 448: 2^-24 relative, 2^-150 where subnormal;
    1 where that rounds to 0.  A code is monotone in h, so it lies between the codes of the two
    ends of h / s, which the quotient's rounding widens by 2^-24."""
    x64 = F.bf16_to_f32(x).astype(np.float64)
    rows, cols = x64.shape[0], x64.shape[1] // 2
    h = moe.swiglu(x64)
    dh = (4 * np.abs(x64[:, :cols]) + 16) * 2.0 ** -24 * np.abs(h) + 2.0 ** -150
    width = cols if scheme == "fp8_row" else 128
    low = np.maximum(np.abs(h) - dh, 0.0).reshape(rows, -1, width).max(2) / 448.0
    high = (np.abs(h) + dh).reshape(rows, -1, width).max(2) / 448.0
    s = q.scales.double().cpu().numpy().reshape(rows, -1)
    near = (s >= low * (1 - 2.0 ** -24) - 2.0 ** -150) & (s <= high * (1 + 2.0 ** -24) + 2.0 ** -150)
    one = (s == 1.0) & (low <= 2.0 ** -150)
    assert ((s > 0) & (near | one)).all(), f"scales off, first at {tuple(np.argwhere(~(near | one))[0])}"
    wide = np.repeat(s, width, axis=1)
    ends = [(h + sign * dh) / wide for sign in (-1, 1)]
    ends = [v + sign * 2.0 ** -24 * np.abs(v) for sign, v in zip((-1, 1), ends)]
    first, last = (F.e4m3_decode(F.e4m3_encode(v)) for v in ends)
    got = F.e4m3_decode(q.codes.cpu().numpy())
    ok = (got >= first) & (got <= last)   # false for a NaN
    assert ok.all(), f"{int((~ok).sum())} codes off, first at {tuple(np.argwhere(~ok)[0])}"


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
@pytest.mark.parametrize("cols", [128, 640, 2304, 9088])
def test_swiglu_far_gates(scheme, cols):
    """Gates so far below zero that 1 + exp(-g) leaves fp32, with up values that bring the product
    back into it: silu(-90) 1e6 = -7e-32."""
    rng = np.random.default_rng(cols)
    rows = 24
    g = rng.uniform(-95.0, -75.0, (rows, cols))
    u = rng.standard_normal((rows, cols)) * 1e6
    g[6:12] = rng.uniform(-199.0, -80.0, (6, cols))
    u[6:12] = rng.choice([-1.0, 1.0], (6, cols)) * np.exp(rng.uniform(40.0, 88.0, (6, cols)))
    g[12:18] = rng.uniform(-130.0, 5.0, (6, cols))          # near and far gates in one row
    u[12:18] *= 1e-3
    g[18] = -300.0                                           # 0 for any finite up value
    g[19, ::2] = -3e38
    g[20], u[20] = -90.0, 1e6
    g[21], u[21] = -88.0, 1.0
    g[22:] = rng.uniform(-110.0, -85.0, (2, cols))           # subnormal h
    u[22:] = rng.standard_normal((2, cols))
    x = F.f32_to_bf16_rne(np.concatenate([g, u], axis=1).astype(np.float32))
    q = pql.swiglu_quantize(up(x), scheme)
    check_swiglu_everywhere(x, scheme, q)
    assert (q.scales.reshape(rows, -1)[18] == 1).all() and not (q.codes[18] & 0x7F).any()
    assert (q.scales.reshape(rows, -1)[20] < 1e-33).all() and ((q.codes[20] & 0x7F) == 0x7E).all()


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
@pytest.mark.parametrize("cols", [128, 384, 2176, 8320])
def test_swiglu_subnormal_scales(scheme, cols):
    """Largest |h| of n 2^-149: the scale is n / 448 rounded to whole steps of 2^-149, so a quotient
    reaches n, well past 448 (n = 656: scale 1 step, quotient 656): the code saturates there, as every
    cast does."""
    rng = np.random.default_rng(cols)
    tops = np.array([1, 200, 224, 228, 300, 448, 480, 600, 656, 672, 1000, 1120, 1360, 2000, 5000, 20000])
    g = np.full((len(tops), cols), 2.0 ** -70)               # silu(g) = 2^-71 exactly, to fp32
    n = tops[:, None] * rng.uniform(-1.0, 1.0, (len(tops), cols))
    n[:, ::128] = tops[:, None]
    x = F.f32_to_bf16_rne(np.concatenate([g, n * 2.0 ** -78], axis=1).astype(np.float32))
    q = pql.swiglu_quantize(up(x), scheme)
    check_swiglu_everywhere(x, scheme, q)
    assert ((q.codes & 0x7F) != 0x7F).all()


# ---------------------------------------------------------------- grouped products
KERNELS = [   # a shape for each kernel
    ("fp8_row", "stream<1", 5, 2, 64, 200, 256), ("fp8_block128", "stream<1", 5, 2, 64, 256, 256),
    ("fp8_row", "stream<1", 40, 3, 30, 200, 256), ("fp8_block128", "stream<1", 40, 3, 30, 256, 256),
    ("fp8_row", "stream<4", 20, 2, 4, 264, 384), ("fp8_block128", "stream<4", 20, 2, 4, 256, 384),
    ("fp8_row", "tile<128", 300, 2, 5, 1401, 256), ("fp8_block128", "tile<128", 300, 2, 5, 1408, 256),
    ("fp8_row", "tile<256", 1350, 2, 9, 8190, 256), ("fp8_block128", "tile<256", 1350, 2, 9, 8064, 256),
]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("scheme,kernel,T,k,E,N,K", KERNELS)
def test_no_kernel_follows_a_wild_plan(scheme, kernel, T, k, E, N, K, gather):
    """Offsets and orders of any value: the call ends and writes nothing outside the result."""
    assert pql.moe_kernel_name(scheme, T, k, E, N, K, gather) == f"k_moe_{kernel}, {scheme}>"
    rng = np.random.default_rng(N)
    a = pql.quantize(torch.randn(T if gather else T * k, K, device=DEV).bfloat16(), scheme)
    w = pql.quantize(torch.randn(E * N, K, device=DEV).bfloat16(), scheme, "weight")
    plan = pql.moe_plan(torch.zeros(T, k, dtype=torch.int32, device=DEV), E)
    big = np.iinfo(np.int32)
    overlapping = np.where(np.arange(E + 1) % 2, big.max, big.min)
    for offsets in (rng.integers(big.min, big.max, E + 1), rng.integers(-5, T * k + 5, E + 1), overlapping,
                    np.full(E + 1, big.max), np.full(E + 1, big.min), np.arange(E + 1)[::-1] * 7):
        plan.offsets.copy_(torch.from_numpy(offsets.astype(np.int32)))
        plan.order.copy_(torch.from_numpy(rng.integers(big.min, big.max, T * k).astype(np.int32)))
        wide = torch.full((T * k + 300, N + 6), 7.0, device=DEV).bfloat16()
        pql.moe_qgemm(a, w, plan, gather=gather, out=wide[:T * k, 3:3 + N])
        wide[:T * k, 3:3 + N] = 7.0
        assert (wide == 7.0).all()


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
@pytest.mark.parametrize("kernel,T,E,N,K", [("tile<256", (1 << 20) - 20, 2, 1024, 4096), ("tile<128", 65535, 2, 256, 65536),
                                            ("stream<4", 65536, 2, 256, 65536)])
def test_gathered_activation_at_the_32_bit_border(scheme, kernel, T, E, N, K):
    """Tiles gather by 32-bit offsets up to an activation of 2^32 - 2^16 bytes; one row more and the
    stream takes it.  Codes of 0, +-1 and +-2 and scales of 1, 2 and 4: every sum is a whole number
    below 2^24, exact in any order, so sampled rows must equal their rounding to bf16."""
    assert pql.moe_kernel_name(scheme, T, 1, E, N, K, True) == f"k_moe_{kernel}, {scheme}>"
    g = torch.Generator(device=DEV).manual_seed(K)
    block = scheme == "fp8_block128"
    table = torch.zeros(64, dtype=torch.uint8, device=DEV)
    table[:4] = torch.tensor([0x38, 0x40, 0xB8, 0xC0], dtype=torch.uint8, device=DEV)   # 1, 2, -1, -2

    def operand(role, rows):
        codes = torch.empty(rows, K, dtype=torch.uint8, device=DEV)
        for r in range(0, rows, 4096):
            part = codes[r:r + 4096]
            part.copy_(table[torch.randint(0, 64, part.shape, device=DEV, generator=g)])
        shape = (rows,) if not block else (rows, K // 128) if role == "activation" else (rows // 128, K // 128)
        return pql.QTensor(scheme, role, rows, K, codes, 2.0 ** torch.randint(0, 3, shape, device=DEV, generator=g).float())

    a, w = operand("activation", T), operand("weight", E * N)
    ids = torch.randint(0, E, (T, 1), dtype=torch.int32, device=DEV, generator=g)
    plan = pql.moe_plan(ids, E)
    c = pql.moe_qgemm(a, w, plan, gather=True)
    value = torch.from_numpy(F.e4m3_decode(np.arange(256, dtype=np.uint8))).to(DEV)
    offsets = plan.offsets.tolist()
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        p = torch.cat([torch.tensor([lo, lo + 1, hi - 2, hi - 1], device=DEV),
                       torch.randint(lo, hi, (24,), device=DEV, generator=g)])
        r = plan.order[p].long()
        s = a.scales[r].double()
        A = value[a.codes[r].long()] * (s.repeat_interleave(128, 1) if block else s[:, None])
        mine = slice(e * N, (e + 1) * N)
        s = w.scales[mine].double()[:, None] if not block else \
            w.scales[e * (N // 128):(e + 1) * (N // 128)].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        want = A @ (value[w.codes[mine].long()] * s).t()
        assert want.abs().max() < 1 << 24
        assert torch.equal(c[p], want.float().bfloat16())


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
def test_a_crowded_expert_in_the_stream(scheme):
    """Every token's first choice is one expert of 256, the second is spread: the streaming kernel walks
    the crowded expert's 512 rows in passes of 16 beside experts of a few rows and empty ones."""
    T, k, E, N, K = 512, 2, 256, 256, 256
    rng = np.random.default_rng(3)
    ids = np.stack([np.full(T, 200), rng.integers(0, 150, T)], axis=1)
    assert pql.moe_kernel_name(scheme, T, k, E, N, K, True) == f"k_moe_stream<1, {scheme}>"
    plan = pql.moe_plan(torch.from_numpy(ids.astype(np.int32)).to(DEV), E)
    offsets, order = plan.offsets.cpu().numpy(), plan.order.cpu().numpy()
    assert offsets[201] - offsets[200] == T
    a, w = exact_operand(scheme, "activation", T, K, 1), exact_operand(scheme, "weight", E * N, K, 2)
    c = pql.moe_qgemm(pql.from_numpy(a, DEV), pql.from_numpy(w, DEV), plan, gather=True)
    c64, _ = moe.gemm(a, w, offsets, order, k, True)
    check_gemm_exact(down(c), c64, f"crowded {scheme}")


# ---------------------------------------------------------------- route
def check_route_rows(x, k, rows, **kw):
    """The kernel on all of ``x``, the oracle on ``rows``: ids equal, weights within what the kernel's
    arithmetic allows.  A score s = exp(d) / z of the distance d = x - max is off by |d| (the
    rounding of d), 2 (the exponential), 40 (z: the terms' 2.23 |d| + 2 with a mean |d| below ln 1024, 22
    roundings) and 1 (the quotient) units of 2^-24; a sigmoid by less; a weight of renormalized
    scores by that and the weighted mean of the others', 1 for its own rounding and half a step of
    the subnormal grid.  Scores below 2^-100 are formed in 64 bits, with no error to speak of."""
    bias = kw.get("bias")
    ids, w = pql.moe_route(x, k, **kw)
    x64 = x[rows].double().cpu().numpy()
    want_ids, want_w = moe.route(x64, k, **{**kw, "bias": None if bias is None else bias.cpu().numpy()})
    assert np.array_equal(ids[rows].cpu().numpy(), want_ids)
    got = w[rows].double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want_w))
    top = np.where(x64 < np.inf, x64, -np.inf).max(1, keepdims=True)
    d = np.abs(np.take_along_axis(x64, np.maximum(want_ids, 0), 1) - np.where(top > -np.inf, top, 0.0))
    d = np.where((want_ids >= 0) & (d < 70.0), d, 0.0) * (kw.get("score", "softmax") == "softmax")
    if kw.get("renormalize", True):
        total = np.abs(want_w).sum(1, keepdims=True)
        d = d + (np.abs(want_w) * d).sum(1, keepdims=True) / np.where(total > 0, total, 1.0) + 43
    ok = np.abs(got - want_w) <= (d + 44) * 2.0 ** -24 * np.abs(want_w) + 2.0 ** -150
    assert ok[~np.isnan(want_w)].all(), f"{int((~ok).sum())} weights off"


@pytest.mark.parametrize("k", [17, 31, 32])
@pytest.mark.parametrize("E,n,top", [(64, 4, 3), (128, 8, 4), (250, 10, 5), (512, 8, 3), (1000, 4, 1)])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("sigmoid", True), ("softmax", True)])
def test_route_more_results_than_lanes(E, n, top, k, score, biased):
    """Many tokens, so 16 or 32 lanes each, and up to 32 experts per token: a lane of 16 keeps a second
    result, and with a bias no lane is left for a further candidate."""
    T = 2061
    g = torch.Generator().manual_seed(E * k)
    x = torch.randn(T, E, generator=g).to(DEV)
    x[7, E // 2:] = -float("inf")
    x[8, 3:] = -float("inf")                                 # fewer experts than results
    x[9, 5] = float("nan")
    bias = (0.1 * torch.randn(E, generator=g)).to(DEV) if biased else None
    rows = torch.cat([torch.arange(24), torch.randint(0, T, (60,), generator=g), torch.arange(T - 9, T)]).to(DEV)
    check_route_rows(x, k, rows, score=score, bias=bias)
    check_route_rows(x, k, rows, score=score, bias=bias, n_groups=n, top_groups=top, renormalize=False, scale=2.5)


@pytest.mark.parametrize("T", [40, 2100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_weights_beside_the_lowest_value(T, score, biased):
    """Masks of the type's lowest value, and logits far from the row's largest."""
    E, k = 48, 12
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, E, generator=g)
    low = torch.finfo(torch.float32).min
    x[0::8, ::2] = low
    x[1::8, 6:] = low                                        # fewer real logits than results
    x[2::8] = low
    x[3::8] *= 30.0
    x[4::8] *= 1000.0
    x[5::8, 1:] = -float("inf")
    x[6::8] *= 1e-30
    bias = (0.1 * torch.randn(E, generator=g)).to(DEV) if biased else None
    rows = torch.arange(0, T, max(1, T // 104), device=DEV)
    rows = torch.cat([rows, torch.arange(16, device=DEV)])
    for renormalize in (True, False):
        check_route_rows(x.to(DEV), k, rows, score=score, bias=bias, renormalize=renormalize)


@pytest.mark.parametrize("T", [300, 2100])
@pytest.mark.parametrize("score,spread", [("sigmoid", 1e-4), ("softmax", 1e-2)])
@pytest.mark.parametrize("level", [3.0, 25.0, 100.0, -1000.0, 3e4, 4e6])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_route_groups_of_large_choices(T, score, spread, level, group_score):
    """Biases that leave few of a choice's bits to the score: the choices, and sums of two, are closer
    than fp32 tells apart, and the order has to be that of 64 bits."""
    E = 128
    g = torch.Generator().manual_seed(T)
    x = (spread * torch.randn(T, E, generator=g)).to(DEV)
    bias = torch.full((E,), level, device=DEV)
    rows = torch.cat([torch.arange(100), torch.arange(T - 20, T)]).to(DEV)
    check_route_rows(x, 6, rows, score=score, bias=bias, n_groups=8, top_groups=3, group_score=group_score)


# ---------------------------------------------------------------- plan
@pytest.mark.parametrize("T,k,E", [(100, 4, 16), (5000, 4, 33), (80000, 8, 60)])
def test_plan_with_the_callers_workspace(T, k, E):
    ids = torch.randint(-1, E + 1, (T, k), dtype=torch.int32, device=DEV, generator=torch.Generator(device=DEV).manual_seed(T))
    want = pql.moe_plan(ids, E)
    need = pql._plan_workspace(T, k, E)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    got = pql.moe_plan(ids, E, workspace=ws)
    again = pql.moe_plan(ids, E, workspace=ws)                # dirty from the first
    for f in ("offsets", "order", "slots"):
        assert torch.equal(getattr(got, f), getattr(want, f)) and torch.equal(getattr(again, f), getattr(want, f))
    assert (ws[need:] == 0x5A).all()
    if need:
        with pytest.raises(ValueError, match="workspace"):
            pql.moe_plan(ids, E, workspace=ws[:need - 1])
        with pytest.raises(ValueError, match="aligned"):
            pql.moe_plan(ids, E, workspace=ws[8:])
    with pytest.raises(ValueError, match="workspace"):
        pql.moe_plan(ids, E, workspace=torch.empty(need, dtype=torch.uint8))


# ---------------------------------------------------------------- together
def _layer(scheme, E, hidden, width, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w_in = (0.05 * torch.randn(E * 2 * width, hidden, device=DEV, generator=g)).bfloat16()
    w_out = (0.05 * torch.randn(E * hidden, width, device=DEV, generator=g)).bfloat16()
    return pql.quantize(w_in, scheme, "weight"), pql.quantize(w_out, scheme, "weight")


SIZES = [(3, 2, 64), (300, 2, 8), (2400, 4, 130), (9000, 2, 6)]   # the streams, tiles of 128 and of 256 rows


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
@pytest.mark.parametrize("T,k,E", SIZES)
def test_layers_at_once(scheme, T, k, E):
    """Two layers on two streams at the same time, several times over: each gives what it gives alone."""
    hidden, width = 512, 768
    wi, wo = _layer(scheme, E, hidden, width, 1)
    inputs = []
    for seed in (1, 2):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x = torch.randn(T, hidden, device=DEV, generator=g).bfloat16()
        inputs.append((x, torch.randn(T, E, device=DEV, generator=g)))

    def layer(x, logits):
        ids, weights = pql.moe_route(logits, k)
        return pql.moe_mlp(x, ids, weights, wi, wo, E, add=x)

    want = [layer(*i) for i in inputs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for s, i, out in zip(streams, inputs, got):
            with torch.cuda.stream(s):
                out.append(layer(*i))
    torch.cuda.synchronize()
    for out, w in zip(got, want):
        assert all(torch.equal(o, w) for o in out)


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
@pytest.mark.parametrize("T,k,E", SIZES)
def test_layer_replayed_with_other_groups(scheme, T, k, E):
    """Captured once; the replays see other group sizes, crowded and empty experts among them."""
    hidden, width = 512, 768
    wi, wo = _layer(scheme, E, hidden, width, 3)
    x, logits = torch.zeros(T, hidden, device=DEV).bfloat16(), torch.zeros(T, E, device=DEV)

    def layer():
        ids, weights = pql.moe_route(logits, k)
        return pql.moe_mlp(x, ids, weights, wi, wo, E)

    def fill(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x.copy_(torch.randn(T, hidden, device=DEV, generator=g))
        logits.copy_(torch.randn(T, E, device=DEV, generator=g))
        if seed == 2:
            logits[:, E // 2] += 50.0                          # everybody's first choice
        if seed == 3:
            logits[:, 3:] = -float("inf")                      # three experts take all
        if seed == 4:
            logits[T // 2:] = -float("inf")                    # no expert for half of the tokens

    fill(1)
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for seed in (2, 3, 4, 1, 2):
        fill(seed)
        want = layer().clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and out.isfinite().all()


@pytest.mark.parametrize("scheme", ["fp8_row", "fp8_block128"])
def test_layer_of_no_tokens_and_of_no_local_experts(scheme):
    wi, wo = _layer(scheme, 2, 128, 256, 1)
    none = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    assert pql.moe_mlp(torch.empty(0, 128, device=DEV).bfloat16(), none, none.float(), wi, wo, 2).shape == (0, 128)
    x = torch.randn(33, 128, device=DEV).bfloat16()
    ids = torch.full((33, 2), 5, dtype=torch.int32, device=DEV)   # all on other ranks
    out = pql.moe_mlp(x, ids, torch.ones(33, 2, device=DEV), wi, wo, 2, add=x)
    assert torch.equal(out, x)
