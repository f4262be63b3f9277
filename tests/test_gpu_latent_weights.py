"""Latent decode: a long tail of small weights beside a large one, against float64.  The requirements
here do not depend on how the kernel holds its weights:

* a value that only the tail has comes out within 1 % where the tail's weights are at least 2^-19 of the
  largest: the output's bf16 rounding is 2^-8 of it, so that 0.6 % is left for weights and scores;
* every output is within 2^-8 of its own size (bf16) plus 2^-9 of the row's largest, whatever the weights.

(A score here is one product, q exact in two e4m3 terms, so its error is fp32's: below 2^-18.)
"""
import numpy as np
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from oracle import latent as olat
from test_gpu_latent import dev, f64  # noqa: F401
from workloads import bf16_bits, latent_inputs

pytestmark = pytest.mark.gpu

H, L, PS = 64, 64, 64


def sink_and_tail(dev, n, sink_key, zeros, fp8, spread=0.0):  # noqa: F811
    """n entries: entry 0 has the largest weight and value 1 in channel 2; the others key -1 and value 1 in
    channel 1; those in `zeros` are rows of zeros.  Head h's tail has weights 2^-(8 + h/4) of the first
    entry's (times a factor of up to 2^spread).  Returns got, want [H, L], exponents."""
    inp = latent_inputs([n], L, 0, PS, seed=91)
    g = torch.Generator().manual_seed(92)
    c = torch.zeros((n, L))
    c[:, 0] = -1.0 + spread * (torch.rand(n, generator=g) - 0.5) / 8
    c[:, 1] = 1.0
    c[:, 3:] = (0.4 * torch.randn((n, L - 3), generator=g)).clamp(-1, 1)
    c[0] = 0.0
    c[0, 0], c[0, 2] = sink_key, 1.0
    c[zeros] = 0.0
    inp.latent[:] = c.to(torch.bfloat16)
    rows, scale = inp.pool(fp8)
    pool = spa.LatentPool(rows.to(dev), inp.block_table.to(dev), 0, scale.to(dev) if fp8 else None)
    suffix = "_fp8" if fp8 else ""
    getattr(spa, "sparse_attn_latent_write" + suffix)(inp.latent.to(dev), None, inp.positions.to(dev), pool)
    exponents = 8 + np.arange(H) / 4
    q = torch.zeros((1, H, L))
    q[0, :, 0] = torch.from_numpy(exponents * np.log(2) / (1 + sink_key))
    q = q.to(torch.bfloat16)
    pos = torch.tensor([n - 1], dtype=torch.int32)
    out = getattr(spa, "sparse_attn_latent_decode" + suffix)(q.to(dev), None, pool, pos.to(dev), scale=1.0)
    assert spa.sparse_attn_paged_check_errors() == 0
    stored = pool.rows.cpu().numpy() if fp8 else bf16_bits(pool.rows.cpu())
    want, _ = olat.decode(f64(q), np.zeros((1, H, 0)), pos.numpy(), None, inp.block_table, stored, page_size=PS,
                          scale=1.0, fp8=fp8, row_scale=pool.scale.cpu().numpy() if fp8 else None)
    return f64(out[0]), want[0][0], exponents


CASES = {
    "50000": dict(n=50000, sink_key=1.0, zeros=[]),
    "131000": dict(n=131000, sink_key=1.0, zeros=[]),
    "100000_a_row_of_zeros": dict(n=100000, sink_key=1.0, zeros=[1]),
    # the sink's score is that of a row of zeros too
    "100000_rows_of_zeros_score_high": dict(n=100000, sink_key=0.0, zeros=[1, 2, 77, 40000]),
    "60000_spread": dict(n=60000, sink_key=1.0, zeros=[5], spread=1.0),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", sorted(CASES))
def test_a_tail_of_small_weights_counts(dev, case, fp8):  # noqa: F811
    got, want, exponents = sink_and_tail(dev, fp8=fp8, **CASES[case])
    err = np.abs(got - want)
    near = exponents <= 19
    rel = err[near, 1] / want[near, 1]
    assert rel.max() <= 0.01, (case, fp8, exponents[near][rel.argmax()], rel.max())
    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * np.abs(want).max(1, keepdims=True)
    assert np.all(err <= bound), (case, fp8, (err / bound).max(1))


def test_rows_of_zeros_alone(dev):  # noqa: F811
    """Nothing but rows of zeros, some whose scale is 1 and one whose codes are all minus zero: zeros."""
    inp = latent_inputs([150], 64, 16, 16, seed=93)
    inp.latent[:] = 0.0
    inp.rope[:] = 0.0
    inp.latent[7], inp.rope[7] = -0.0, -0.0
    rows, scale = inp.pool(True)
    pool = spa.LatentPool(rows.to(dev), inp.block_table.to(dev), 16, scale.to(dev))
    spa.sparse_attn_latent_write_fp8(inp.latent.to(dev), inp.rope.to(dev), inp.positions.to(dev), pool)
    q = torch.randn((1, 8, 80), generator=torch.Generator().manual_seed(94)).to(torch.bfloat16).to(dev)
    out = spa.sparse_attn_latent_decode_fp8(q[..., :64], q[..., 64:], pool,
                                            torch.tensor([149], dtype=torch.int32, device=dev), scale=1.0)
    assert bool((out == 0).all())


def test_rows_whose_scale_is_one_but_hold_values(dev):  # noqa: F811
    """Rows with a largest value of exactly 448, in the first or the last place of the row, beside rows of
    zeros: only the latter count as zeros."""
    n, R = 200, 16
    inp = latent_inputs([n], 64, R, 16, seed=95)
    inp.latent[:] = 0.0
    inp.rope[:] = 0.0
    inp.latent[10:60, 0] = 448.0
    inp.latent[60:90, 63] = -448.0
    inp.rope[90:120, R - 1] = 448.0
    rows, scale = inp.pool(True)
    pool = spa.LatentPool(rows.to(dev), inp.block_table.to(dev), R, scale.to(dev))
    spa.sparse_attn_latent_write_fp8(inp.latent.to(dev), inp.rope.to(dev), inp.positions.to(dev), pool)
    q = torch.zeros((1, 3, 64 + R), dtype=torch.bfloat16)
    q[0, 0, 0], q[0, 1, 63], q[0, 2, 64 + R - 1] = 2.0 ** -8, 2.0 ** -8, 2.0 ** -8
    pos = torch.tensor([n - 1], dtype=torch.int32)
    out = spa.sparse_attn_latent_decode_fp8(q[..., :64].to(dev), q[..., 64:].to(dev), pool, pos.to(dev),
                                            scale=1.0)
    want, _ = olat.decode(f64(q[..., :64]), f64(q[..., 64:]), pos.numpy(), None, inp.block_table,
                          pool.rows.cpu().numpy(), page_size=16, scale=1.0, fp8=True,
                          row_scale=pool.scale.cpu().numpy())
    o = want[0][0]
    assert np.all(np.abs(f64(out[0]) - o) <= 2.0 ** -7 * np.abs(o) + 2.0 ** -9 * np.abs(o).max(1, keepdims=True))
