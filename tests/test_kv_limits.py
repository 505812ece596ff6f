"""The borders of what the calls around the cache of keys and values accept: given scales in fp32, workspaces,
sizes.  No GPU needed."""
import math

import pytest
import torch

import precision_quantized_linear_amd as pql


# ---------------------------------------------------------------- given scales
@pytest.mark.parametrize("scale", [1e-50, 1e39, 2.0 ** -150, 3.4028236e38, 1e400, -1.0, math.nan])
def test_scales_that_fp32_makes_zero_or_infinite(scale):
    for kw in (dict(k_scale=scale, v_scale=1.0), dict(k_scale=1.0, v_scale=scale)):
        with pytest.raises(ValueError, match="fp8_tensor needs"):
            pql.kv_cache(2, 16, 1, 64, "fp8_tensor", device="cpu", **kw)


@pytest.mark.parametrize("scale", [2.0 ** -149, 2.0 ** -126, 1, 3.4028235e38, torch.tensor(0.5)])
def test_scales_at_the_ends_of_fp32(scale):
    cache = pql.kv_cache(2, 16, 1, 64, "fp8_tensor", device="cpu", k_scale=scale, v_scale=scale)
    assert 0 < cache.k_scales.item() < math.inf and cache.k_scales.item() == cache.v_scales.item()


# ---------------------------------------------------------------- workspaces
@pytest.mark.parametrize("H,Hk,T,B,rows", [(32, 32, 4096, 1, 128), (128, 128, 4096, 1, 128), (64, 64, 64, 64, 16), (256, 64, 1024, 64, 32)])
def test_a_workspace_holds_no_more_ranges_than_there_can_be(H, Hk, T, B, rows):
    """Contexts are cut so that fewer than 2 target / Hk ranges of a head need a place; the target is below 1.5 rounds of
    two workgroups per CU with many rows, at most three rounds of three with few."""
    width = 512
    name = pql.kv_kernel_name("fp8_row", T, H, Hk, 128, B, width, 16)
    assert ("tile" if rows == 128 else f"<{rows}>") in name and "join" in name
    places = pql.kv_attention_workspace("fp8_row", T, H, Hk, 128, B, width, 16) / (Hk * rows * (128 + 4) * 4)
    assert 0 < places <= 2 * ((767 if rows == 128 else 9 * 256) // Hk + 1)


# ---------------------------------------------------------------- sizes: the last one taken and the first refused
# Calls that pass the checks of sizes are refused for their NULL operands: nothing is ever launched.
NULL = "must be non-NULL"


def refusal(status):
    assert status == pql.PQL_ERR_INVALID_ARGUMENT
    return pql.lib().pql_last_error().decode()


@pytest.mark.parametrize("D,T,H,fits", [(64, 1 << 28, 1, True), (64, (1 << 28) + 1, 1, False), (64, 1 << 20, 1 << 8, True),
                                        (64, 1 << 20, (1 << 8) + 1, False), (256, 1 << 26, 1, True), (256, 1 << 25, 3, False),
                                        (16, 1 << 30, 1, True), (16, (1 << 30) + 1, 1, False), (1024, 1 << 24, 1, True),
                                        (1024, 1 << 23, 3, False)])
def test_rope_sizes(D, T, H, fits):
    text = refusal(pql.lib().pql_rope(0, None, T, H, D, H * D, D, 1 << 20, 1 << 20, 16, 1.0, None, H * D, D, None))
    assert (NULL in text) == fits and ("too large" in text) != fits


@pytest.mark.parametrize("D,n,Hk,fits", [(64, 1 << 27, 2, True), (64, (1 << 27) + 1, 2, False), (256, 1 << 20, 64, True),
                                         (256, (1 << 20) + 1, 64, False)])
def test_append_and_read_sizes(D, n, Hk, fits):
    st = (Hk * D, D)
    for status in (pql.lib().pql_kv_append(2, None, *st, None, *st, n, None, 0, None, None, 0, 1.0, None, None, None, None,
                                           4, 16, Hk, D, None),
                   pql.lib().pql_kv_read(2, None, None, None, None, 4, 16, Hk, D, None, n, None, *st, None, *st, None)):
        text = refusal(status)
        assert (NULL in text) == fits and ("too large" in text) != fits


@pytest.mark.parametrize("T,H,Hk,D,B,fits", [
    (1, 65535, 1, 64, 1, True), (1, 65536, 1, 64, 1, False), (1 << 20, 256, 8, 64, 1, True), ((1 << 20) + 1, 256, 8, 64, 1, False),
    (1 << 20, 15, 15, 64, 1 << 20, True), (1 << 20, 16, 16, 64, 1 << 20, False), (1, 1, 1, 256, 1 << 20, True),
    (1, 1, 1, 256, (1 << 20) + 1, False),
])
def test_attention_sizes(T, H, Hk, D, B, fits):
    assert bool(pql.kv_kernel_name("fp8_row", T, H, Hk, D, B, 1, 16)) == fits
    if fits:
        pql.kv_attention_workspace("fp8_row", T, H, Hk, D, B, 1, 16)
    else:
        with pytest.raises(ValueError):
            pql.kv_attention_workspace("fp8_row", T, H, Hk, D, B, 1, 16)


def test_batch_sizes():
    L = pql.lib()
    assert NULL in refusal(L.pql_kv_slots(None, None, None, 1 << 20, 1, 1 << 20, 16, 4, None, None, None))
    assert "ldp must" in refusal(L.pql_kv_slots(None, None, None, 1 << 20, 1, (1 << 20) + 2, 16, 4, None, None, None))
    assert NULL in refusal(L.pql_kv_slots(None, None, None, 1, 1 << 26, 1 << 26, 16, 4, None, None, None))
    assert "width" in refusal(L.pql_kv_slots(None, None, None, 1, (1 << 26) + 1, 1 << 27, 16, 4, None, None, None))
    assert "B must" in refusal(L.pql_kv_slots(None, None, None, (1 << 20) + 1, 1, 1, 16, 4, None, None, None))
    assert NULL in refusal(L.pql_kv_slots(None, None, None, 1, 1, 1, 16, (1 << 31) - 1, None, None, None))
    assert "T must" in refusal(L.pql_kv_slots(None, None, None, 1, 1, 1, 16, 1 << 31, None, None, None))


# ---------------------------------------------------------------- rotary tables
@pytest.mark.parametrize("scaling", [
    dict(type="yarn", factor=2.0, original=math.inf), dict(type="yarn", factor=2.0, original=4096, fast=math.inf),
    dict(type="yarn", factor=2.0, original=4096, attention=math.nan), dict(type="yarn", factor=2.0, original=4096, attention=math.inf),
    dict(type="yarn", factor=2.0, original=4096, attention=1e39), dict(type="ntk", factor=1e300),
])
def test_stretching_that_leaves_the_numbers_range(scaling):
    """Refused by name where the table is made, not as an overflow there or by a later call."""
    with pytest.raises(ValueError, match=scaling["type"] + " scaling needs"):
        pql.rope_freqs(64, scaling=scaling)
