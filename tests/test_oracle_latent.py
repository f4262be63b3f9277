"""The latent-attention oracle against independent restatements (CPU only)."""
import math

import numpy as np
import pytest

from oracle import bf16_to_f64, e4m3_to_f64, latent
from workloads import bf16_bits, latent_inputs

ALL_CODES = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)


def nearest(x):
    """The e4m3 value nearest to x by search over every finite code (ties to the even code)."""
    v = e4m3_to_f64(ALL_CODES)
    d = np.abs(v - x)
    best = np.flatnonzero(d == d.min())
    even = [i for i in best if ALL_CODES[i] % 2 == 0]
    return v[(even or list(best))[0]]


def test_quantised_rows_are_nearest_codes_and_the_low_code_halves_what_is_left():
    inp = latent_inputs([6], 64, 16, 4, seed=1)
    for t in range(6):
        x = bf16_to_f64(np.concatenate([bf16_bits(inp.latent[t]), bf16_bits(inp.rope[t])]))
        codes, scale = latent.quantize_row(x.astype(np.float32), 16)
        assert scale == np.float32(np.float32(np.abs(x).max()) / np.float32(448))
        y = (x.astype(np.float32) / scale).astype(np.float64)
        v = e4m3_to_f64(codes)
        assert all(v[i] == nearest(y[i]) for i in range(80))
        assert all(v[80 + i] == nearest(y[64 + i] - v[64 + i]) for i in range(16))
        back = latent.row_values(codes[None], 64, 16, fp8=True, scale=np.array([scale]))[0]
        # half a step: 2^-4 of the value; the rotary part 2^-4 of what the first code left
        assert np.all(np.abs(back[:64] - x[:64]) <= 2.0 ** -4 * np.abs(x[:64]) + scale * 2.0 ** -10)
        assert np.all(np.abs(back[64:] - x[64:]) <= 2.0 ** -8 * np.abs(x[64:]) + scale * 2.0 ** -10)


def test_zero_row_and_no_rotary_part():
    codes, scale = latent.quantize_row(np.zeros(72, np.float32), 8)
    assert scale == 1.0 and len(codes) == 80 and not codes.any()
    codes, scale = latent.quantize_row(np.full(64, -3.0, np.float32), 0)
    # the code is -448 and the scale 3 / 448 rounded to binary32 (half a step: 2^-24 of it)
    assert len(codes) == 64 and np.all(np.abs(e4m3_to_f64(codes) * np.float64(scale) + 3.0) <=
                                       3.0 * 2.0 ** -24)


def test_entries_of_a_hand_made_table():
    bt = np.array([[2, -1, 0], [1, 9, 1]])
    at, bad = latent.entries(0, 5, bt, 3, 2)
    assert at.tolist() == [4, 5, 0] and bad            # entries 2 and 3 are unmapped
    assert latent.entries(0, 2, bt, 3, 2)[1] is False
    at, bad = latent.entries(1, 7, bt, 3, 2)           # block 9 is outside, entry 6 past the table
    assert at.tolist() == [2, 3, 2, 3] and bad
    assert latent.entries(2, 1, bt, 3, 2)[1] and len(latent.entries(-1, 1, bt, 3, 2)[0]) == 0


def test_attend_terms_by_hand():
    q = np.array([[1.0, 0.0]])
    k = np.array([[math.log(3.0), 5.0], [0.0, -7.0]])
    v = np.array([[4.0], [-8.0]])
    out, t = latent.attend_terms(q, k, v, 1.0)
    assert np.allclose(t["p"], [[0.75, 0.25]]) and np.allclose(out, 1.0) and np.allclose(t["mass"], 5.0)
    out, t = latent.attend_terms(q, k[:0], v[:0], 1.0)
    assert out.tolist() == [[0.0]]


@pytest.mark.parametrize("fp8", [False, True])
def test_absorbed_equals_expanded(fp8):
    """With k_nope_h = W_uk_h c and v_h = W_uv_h c the two forms are one attention."""
    L, R, H, dn, dv, ps = 64, 16, 3, 24, 16, 4
    lens = [9, 1, 6]
    inp = latent_inputs(lens, L, R, ps, seed=2)
    rows, scale = inp.pool(fp8)
    pool = rows.numpy() if fp8 else bf16_bits(rows)
    sc = scale.numpy() if fp8 else None
    assert not latent.write(bf16_bits(inp.latent), bf16_bits(inp.rope), inp.positions.numpy(),
                            inp.seq_of_token.numpy(), inp.block_table.numpy(), pool, page_size=ps,
                            scale=sc, fp8=fp8)
    rng = np.random.default_rng(3)
    w_uk, w_uv = rng.standard_normal((H, dn, L)) / 8, rng.standard_normal((H, dv, L)) / 8
    T = sum(lens)
    q = rng.standard_normal((T, H, dn + R))
    at = np.concatenate([latent.entries(b, n, inp.block_table, inp.num_blocks, ps)[0]
                         for b, n in enumerate(lens)])
    x = latent.row_values(pool.reshape(inp.num_blocks * ps, -1)[at], L, R, fp8=fp8,
                          scale=None if sc is None else sc[at])
    cu = np.concatenate([[0], np.cumsum(lens)])
    full = latent.prefill(q, np.einsum("tl,hdl->thd", x[:, :L], w_uk), x[:, L:],
                          np.einsum("tl,hdl->thd", x[:, :L], w_uv), cu, cu, scale=0.2)
    ql = np.einsum("thd,hdl->thl", q[..., :dn], w_uk)
    absorbed, err = latent.decode(ql, q[..., dn:], inp.positions.numpy(), inp.seq_of_token.numpy(),
                                  inp.block_table, pool, page_size=ps, scale=0.2, fp8=fp8,
                                  row_scale=sc)
    assert not err
    for t in range(T):
        up = np.einsum("hl,hdl->hd", absorbed[t][0], w_uv)
        assert np.allclose(up, full[t][0], rtol=0, atol=1e-12)


def test_queries_before_the_first_key_see_nothing():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((5, 2, 8)), rng.standard_normal((3, 2, 8)), rng.standard_normal((3, 2, 4))
    res = latent.prefill(q, k, np.zeros((3, 0)), v, [0, 5], [0, 3], scale=1.0)
    assert not res[0][0].any() and not res[1][0].any()
    assert np.allclose(res[2][0], v[0]) and res[4][1]["p"].shape == (2, 3)


def test_quotients_of_the_write_are_the_rounded_ones():
    """x / scale by a correctly rounded reciprocal and one correction, as the e4m3 write works it out, for
    every mantissa of a bf16 x and every scale that a row can have (up to powers of two)."""
    from fractions import Fraction

    def rn(x):                                       # to 24 bits, nearest even
        if x == 0:
            return x
        e = x.numerator.bit_length() - x.denominator.bit_length()
        e -= abs(x) < Fraction(2) ** e
        ulp = Fraction(2) ** (e - 23)
        return round(x / ulp) * ulp

    for m in range(128, 256):
        scale = rn(Fraction(m, 448))
        r = rn(1 / scale)
        for n in range(128, 256):
            x = Fraction(n)
            q = rn(x * r)
            assert rn(q + rn(x - q * scale) * r) == rn(x / scale), (m, n)
