"""Edges of the attention over a paged cache, against the float64 oracle with the bounds of
tests/kv_check.py: values of extreme sizes."""
import numpy as np
import pytest

import precision_quantized_linear_amd as pql
from kv_check import Filled, bf16_bits, check_attention, expected, f64, up16
from oracle import formats as F

pytestmark = pytest.mark.gpu


def run_values(seed, L, new, values, *, H=4, Hk=2, D=128, small=None):
    """One fp8_row sequence of L tokens with the given values [L, Hk, D] and even weights."""
    rng = np.random.default_rng(seed)
    keys = rng.standard_normal((L, Hk, D)) * 0.2
    fill = Filled(rng, "fp8_row", [L], Hk, D, 16, [new], bits=[[bf16_bits(keys), bf16_bits(values)]])
    qb = bf16_bits(rng.standard_normal((new, H, D)))
    q64 = F.bf16_to_f32(qb).astype(np.float64)
    got, lse = pql.kv_attention(up16(qb), fill.cache, fill.starts, fill.lens, fill.pages, return_lse=True)
    check_attention(fill, q64, f64(got), f64(lse), expected(fill, q64), small=L if small is None else small)
    return f64(got)


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
