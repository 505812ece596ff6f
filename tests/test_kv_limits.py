"""The borders of what the calls around the cache of keys and values accept: given scales in fp32.  No GPU needed."""
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
