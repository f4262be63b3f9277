"""Latent attention: scales whose product with log2(e) overflows fp32 are refused (host checks, CPU only)."""
import pytest

import sparse_paged_attention_gb300 as spa
from test_latent_abi import decode, lib, pool, prefill, problem  # noqa: F401

S = spa.SPA_STATUS


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scales_past_the_range_are_refused(lib, sign):  # noqa: F811
    """With such a scale a score of 0 would become NaN (0 times infinity)."""
    for fp8 in (False, True):
        assert decode(lib, pool(), problem(scale=sign * 2.5e38), fp8) == S["SPA_ERR_SHAPE"]
        assert decode(lib, pool(), problem(scale=sign * 2.3e38), fp8) == S["SPA_ERR_CUDA"]   # (no device)
    assert prefill(lib, scale=sign * 2.5e38) == S["SPA_ERR_SHAPE"]
    assert prefill(lib, scale=sign * 2.3e38) == S["SPA_ERR_CUDA"]
