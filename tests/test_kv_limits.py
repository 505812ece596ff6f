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
