"""e4m3 appends of rows so small that a 448th of their maximum is below half of fp32's smallest number, as the
smallest bf16 numbers are times a small amplitude: the scale must not become zero (0 / 0 is a NaN in the cache).

The scale is then 2^-149, and values are multiples of it: two products and a sum are each off by half of it, and a
code by half a step, 2^-4 of the value (whole numbers of at most 224 are no subnormal codes)."""
import numpy as np
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from oracle import e4m3_to_f64
from oracle import latent as olat
from oracle import rotary as orot
from test_gpu_latent import clean_error_word, dev, f64  # noqa: F401

pytestmark = pytest.mark.gpu

D, R, T, PAGE = 64, 16, 12, 16


def tiny():
    """[T, D]: zeros and, in the last R values, a few of the smallest bf16 numbers, one at least."""
    bits = np.zeros((T, D), dtype=np.int16)
    r = np.random.RandomState(1)
    bits[:, D - R:] = r.randint(0, 3, (T, R))
    bits[:, D - R] = 1
    bits[::3, D - R + 1:] = 0
    return torch.from_numpy(bits).view(torch.bfloat16)


def check(got, scale, want):
    assert np.all(scale == 2.0 ** -149), scale
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2 * 2.0 ** -149)


@pytest.mark.parametrize("interleaved", [True, False])
def test_tiny_rows_have_a_scale(dev, interleaved):  # noqa: F811
    x = tiny()
    tab = spa.sparse_attn_rotary_table(R, interleaved=interleaved, scale=2.0 ** -11, device=dev)
    pos = torch.arange(T, dtype=torch.int32)
    want = orot.rotate(f64(x), pos.tolist(), tab.turns.tolist(), start=D - R, interleaved=interleaved, scale=tab.scale)
    assert np.all(np.abs(want).max(1) < 448 * 2.0 ** -150) and np.all(np.abs(want).max(1) > 2.0 ** -149)
    bt = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    kv = spa.PagedPool(torch.zeros((1, PAGE, 2, D), dtype=torch.uint8, device=dev), bt,
                       torch.zeros(PAGE, device=dev), torch.zeros(PAGE, device=dev))
    xd = x.to(dev)
    spa.sparse_attn_paged_kv_append_fp8(xd, xd, pos.to(dev), kv, tab)
    ks = kv.k_scale.cpu().double().numpy()[:T]
    check(e4m3_to_f64(kv.kv[0, :T, 0].cpu().numpy()) * ks[:, None], ks, want)
    lat = spa.LatentPool(torch.zeros((1, PAGE, D + 2 * R), dtype=torch.uint8, device=dev), bt, R,
                         torch.zeros(PAGE, device=dev))
    spa.sparse_attn_latent_append_fp8(torch.zeros_like(xd), xd[:, D - R:], pos.to(dev), lat, tab)
    s = lat.scale.cpu().double().numpy()[:T]
    got = olat.row_values(lat.rows[0, :T].cpu().numpy(), D, R, fp8=True, scale=s)
    check(got, s, np.concatenate([np.zeros((T, D)), want[:, D - R:]], 1))
