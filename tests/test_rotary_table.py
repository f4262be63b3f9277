"""Frequencies scaled for long contexts, against the published ramp written out (CPU only)."""
import math

import numpy as np
import pytest

import sparse_paged_attention_gb300 as spa


def frequencies(table):
    """Radians a position, from turns in 64-bit binary fractions (frequencies of up to 1 are below half a turn)."""
    return table.turns.numpy().astype(np.float64) / 2.0 ** 64 * 2 * math.pi


def yarn(dim, base, factor, length, fast, slow):
    """Pair i keeps its frequency below the pair that turns `fast` times within `length`, is divided by the factor from
    the one on that turns `slow` times, and lies on a straight line between them; the line's ends are whole numbers
    within 0 .. dim - 1."""
    out = []
    ends = [dim * math.log(length / (2 * math.pi * n)) / (2 * math.log(base)) for n in (fast, slow)]
    lo, hi = max(0, math.floor(ends[0])), min(dim - 1, math.ceil(ends[1]))
    for i in range(dim // 2):
        kept = base ** (-2 * i / dim)
        part = 0.0 if i <= lo else 1.0 if i >= hi else (i - lo) / (hi - lo)
        out.append(kept * (1 - part) + kept / factor * part)
    return np.array(out)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("factor", [8.0, 16.0])
@pytest.mark.parametrize("length", [4096, 32768, 65536, 131072, 1 << 20])
@pytest.mark.parametrize("fast,slow", [(32.0, 1.0), (16.0, 2.0)])
def test_yarn_at_long_original_lengths(dim, factor, length, fast, slow):
    base = 10000.0
    table = spa.sparse_attn_rotary_table(dim, base=base, scaling="yarn", factor=factor, original_length=length,
                                         beta_fast=fast, beta_slow=slow, device="cpu")
    got, want = frequencies(table), yarn(dim, base, factor, length, fast, slow)
    # a handful of 64-bit operations, a quotient by 2 pi and its rounding to 2^-64 turns
    np.testing.assert_allclose(got, want, rtol=16 * 2.0 ** -53, atol=2.0 ** -61)
    # a pair that turns more than `slow` times is never divided by the whole factor
    plain = base ** (-2 * np.arange(dim // 2) / dim)
    turning = plain * length / (2 * math.pi) > slow
    assert (got[turning] > 1.0001 * plain[turning] / factor).all()
    assert table.scale == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-15)
