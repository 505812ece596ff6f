"""Edges of the mixture-of-experts operators on the GPU, against the float64 oracle (oracle/moe.py)."""
import numpy as np
import pytest
import torch

import precision_quantized_linear_amd as pql
from oracle import formats as F
from oracle import moe
from test_gpu_moe import up

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
