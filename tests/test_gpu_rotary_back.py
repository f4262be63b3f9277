"""A rotation and its inverse with an amplitude: the inverse turns back and multiplies by the amplitude once more (it
is the rotation's transpose), so that x there and back is the amplitude's square times x."""
import numpy as np
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from oracle import rotary as orot
from test_gpu_latent import clean_error_word, dev, f64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("factor", [1.0, 16.0])
def test_there_and_back(dev, factor, interleaved):  # noqa: F811
    R, D, T, H = 64, 96, 40, 3
    x = torch.randn((T, H, D), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    tab = spa.sparse_attn_rotary_table(R, scaling="yarn", factor=factor, interleaved=interleaved, device=dev)
    m = tab.scale
    assert m == pytest.approx(0.1 * np.log(factor) + 1.0)
    pos = torch.randint(-1000, 1 << 20, (T,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(dev)
    there = spa.sparse_attn_rope(x.to(dev), pos, tab)
    back = f64(spa.sparse_attn_rope(there, pos, tab, inverse=True))
    want = f64(x)
    want[..., D - R:] *= m * m
    # the first result's rounding (2^-8 of a and b) turned back, the second's own, and fp32 in both
    first = m * orot.pair_sizes(f64(there), start=D - R, R=R, interleaved=interleaved)
    assert np.all(np.abs(back - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * 10 * 2.0 ** -24) * 2 * first)
    # its transpose: <y, rope(x)> = <rope_inverse(y), x>
    y = torch.randn((T, H, D), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    turned = f64(spa.sparse_attn_rope(y.to(dev), pos, tab, inverse=True))
    a, b = (f64(y) * f64(there)).sum(-1), (turned * f64(x)).sum(-1)
    slack = 2.0 ** -8 * (np.abs(f64(y) * f64(there)) + np.abs(turned * f64(x))).sum(-1) * 1.01 + 1e-4
    assert np.all(np.abs(a - b) <= slack)
