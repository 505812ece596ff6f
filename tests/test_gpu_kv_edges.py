"""Edges of the attention over a paged cache, against the float64 oracle with the bounds of
tests/kv_check.py: values of extreme sizes, far positions.

Values whose scale lies below 2^-90 are held as weights relative to that, in fp16: a weight (at least 2^7
for the largest) is off by up to 2^-25 beside its relative error, its code is at most 448, and the sum that
divides is at least 2^(7 + 90): 448 2^-122 for each key, `floor` below."""
import numpy as np
import pytest
import torch

import precision_quantized_linear_amd as pql
from kv_check import Filled, bf16_bits, check_attention, expected, f64, up16
from oracle import formats as F
from oracle import kv as okv

pytestmark = pytest.mark.gpu


def run_values(seed, L, new, values, *, H=4, Hk=2, D=128, floor=False):
    """One fp8_row sequence of L tokens with the given values [L, Hk, D] and even weights."""
    rng = np.random.default_rng(seed)
    keys = rng.standard_normal((L, Hk, D)) * 0.2
    fill = Filled(rng, "fp8_row", [L], Hk, D, 16, [new], bits=[[bf16_bits(keys), bf16_bits(values)]])
    qb = bf16_bits(rng.standard_normal((new, H, D)))
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    got, lse = pql.kv_attention(up16(qb), fill.cache, fill.starts, fill.lens, fill.pages, return_lse=True)
    want = expected(fill, q64)
    got = f64(got)
    err = got - want[0]
    if floor:      # what is within the floor counts as none
        got = want[0] + np.sign(err) * np.maximum(np.abs(err) - L * 448 * 2.0 ** -122, 0.0)
    check_attention(fill, q64, got, f64(lse), want, small=L)


# Where the rows of zeros lie among L tokens: before the others, behind them, in every other run of 32 (a
# wave's step), 64 (a key tile) or 512 (a range).
PLACES = {"first": lambda j, L: j < L // 2, "last": lambda j, L: j >= L // 2, "32": lambda j, L: j // 32 % 2 == 0,
          "64": lambda j, L: j // 64 % 2 == 0, "512": lambda j, L: j // 512 % 2 == 0}


@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("L", [300, 3000])
@pytest.mark.parametrize("new", [1, 24, 70])
@pytest.mark.parametrize("size", [1.0, 1e20, 1e34])
def test_rows_of_zeros_beside_large_values(size, new, L, place):
    """A token whose values are zeros keeps its weight whatever the others' sizes: about half of it here."""
    rng = np.random.default_rng(1)
    values = rng.standard_normal((L, 2, 128)) * size
    values[PLACES[place](np.arange(L), L)] = 0.0
    run_values(2, L, new, values)


@pytest.mark.parametrize("L", [300, 3000])
@pytest.mark.parametrize("new", [1, 24, 70])
@pytest.mark.parametrize("sizes", [(1e-26, 1e-28), (1e-30, 1e-30), (1e-33, 0.0), (1e-30, 1.0), (1e-30, 1e34), (1e-38, 1e-39)])
def test_tiny_values(sizes, new, L):
    """Values whose scales lie below 2^-90 keep their size, and their tokens their weight beside large ones."""
    rng = np.random.default_rng(3)
    values = rng.standard_normal((L, 2, 128)) * rng.choice(sizes, (L, 2, 1))
    run_values(4, L, new, values, floor=True)


@pytest.mark.parametrize("L", [300, 3000])
@pytest.mark.parametrize("new", [1, 24, 70])
@pytest.mark.parametrize("scale", [-np.inf, -5.0, -1.0, 0.0, 1e-40, 1e-30, 1.0, 1e38, np.inf])
def test_scales_of_unseen_tokens(scale, new, L):
    """Any scale of a token that no row, or not every row, sees reaches nobody else."""
    rng = np.random.default_rng(5)
    keys, values = (bf16_bits(rng.standard_normal((L, 2, 128))) for _ in "kv")
    fill = Filled(rng, "fp8_row", [L], 2, 128, 16, [new], bits=[[keys, values]])
    qb = bf16_bits(rng.standard_normal((new, 4, 128)))
    fill.cache.v_scales[torch.isnan(fill.cache.v_scales)] = float(scale)
    fill.cache.v_scales[int(fill.pages_np[0, (L - 1) // 16]), :, (L - 1) % 16] = float(scale)   # the last token sees itself
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    want = expected(fill, q64)
    got, lse = pql.kv_attention(up16(qb), fill.cache, fill.starts, fill.lens, fill.pages, return_lse=True)
    rows = np.arange(new - 1)
    check_attention(fill, q64, np.where(np.isfinite(f64(got)), f64(got), 1e300), f64(lse), want, rows=rows, small=L)


# ---------------------------------------------------------------- far positions
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new", [1, 24, 70])
@pytest.mark.parametrize("first", [0, 1, 20, 47, 48, 1 << 29])
def test_windows_of_positions_far_past_the_pages(first, new, causal):
    """A sequence of 2^31 - 1 tokens, all absent but the first 48: the last token's window, of up to
    2^31 - 1 tokens, begins at `first`."""
    rng = np.random.default_rng(6)
    L, held = (1 << 31) - 1, 48
    fill = Filled(rng, "fp8_row", [held], 2, 64, 16, [new])
    fill.lens = torch.tensor([L], dtype=torch.int32, device=fill.lens.device)
    qb = bf16_bits(rng.standard_normal((new, 4, 64)))
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    window = L - first
    seen = np.arange(held)[None] > np.arange(L - new, L)[:, None] - window
    want = okv.attend(q64, fill.k[0], fill.v[0], seen, 64 ** -0.5)
    for w in (window, 1 << 40) if first == 0 else (window,):
        got, lse = pql.kv_attention(up16(qb), fill.cache, fill.starts, fill.lens, fill.pages, causal=causal, window=w,
                                    return_lse=True)
        check_attention(fill, q64, f64(got), f64(lse), want)
