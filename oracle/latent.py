"""Latent attention: the cache's write and read, the absorbed and the expanded form.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain numpy, float64, from the definitions;
shares no code with the CUDA library.

A row x = [c | r]: the latent part c (L values) is key and value of every head, the rotary part r
(R values) belongs to the key.  Slots are those of the paged KV write (``oracle.kv_write.slot_of``).

* e4m3 rows: ``scale = max|x| / 448`` (1 for a zero row), codes ``e4m3(x / scale)``; the rotary
  part has a second, low code ``e4m3(x / scale - high)``.  Scale and quotients are binary32, as they
  decide integer codes; the difference of a binary32 quotient and its code is exact.
* absorbed: ``s_j = scale (q_c . c_j + q_r . r_j)`` over the entries j <= position,
  ``out = sum_j softmax(s)_j c_j``.
* expanded: per head ``k = [k_nope | k_rope]``; query i of a sequence of n_q queries and n_k keys
  sees keys ``j <= i + n_k - n_q``.

Every function that sums also returns what an error bound needs (see ``attend_terms``).
Parity status: the write and the read exact; the attention within bounds derived in the tests.
Pinned by tests/test_oracle_latent.py.
"""
import numpy as np

from .kv_write import E4M3_MAX, e4m3_encode_rne, slot_of
from .sparse_attention import bf16_to_f64, e4m3_to_f64


def quantize_row(x_f32: np.ndarray, rope_dim: int):
    """One binary32 row [c | r] -> (codes [c | high | low], binary32 scale)."""
    x = np.asarray(x_f32, dtype=np.float32)
    amax = np.float32(np.max(np.abs(x)))
    scale = np.float32(amax / np.float32(E4M3_MAX)) if amax > 0 else np.float32(1.0)
    y = (x / scale).astype(np.float32)
    high = e4m3_encode_rne(y)
    if rope_dim == 0:
        return high, scale
    rest = y[-rope_dim:].astype(np.float64) - e4m3_to_f64(high[-rope_dim:])
    return np.concatenate([high, e4m3_encode_rne(rest)]), scale


def row_values(rows, latent_dim: int, rope_dim: int, *, fp8: bool, scale=None) -> np.ndarray:
    """Stored rows [n, width] (uint16 bf16 patterns or uint8 codes, with scales [n]) in float64."""
    if not fp8:
        return bf16_to_f64(rows)
    v = e4m3_to_f64(rows)
    L, R = latent_dim, rope_dim
    r = v[:, L:L + R] + v[:, L + R:L + 2 * R]
    return np.concatenate([v[:, :L], r], 1) * np.asarray(scale, dtype=np.float64)[:, None]


def write(latent_bits, rope_bits, positions, seq_of_token, block_table, pool_rows, *,
          page_size: int, scale=None, fp8: bool) -> bool:
    """Write T tokens' rows in place (pool_rows [num_blocks, page_size, width]); True if one was
    dropped."""
    bt = np.asarray(block_table, dtype=np.int64)
    nb = pool_rows.shape[0]
    flat = pool_rows.reshape(nb * page_size, -1)
    dropped = False
    for t in range(len(positions)):
        b = 0 if seq_of_token is None else int(seq_of_token[t])
        row = slot_of(int(positions[t]), b, bt, nb, page_size)
        if row is None:
            dropped = True
            continue
        bits = np.concatenate([latent_bits[t], rope_bits[t]])
        if fp8:
            flat[row], scale[row] = quantize_row(bf16_to_f64(bits).astype(np.float32),
                                                 len(rope_bits[t]))
        else:
            flat[row] = bits
    return dropped


def entries(b: int, n: int, block_table, num_blocks: int, page_size: int):
    """Pool rows of the entries 0 .. n-1 of sequence b that exist, and whether one does not."""
    bt = np.asarray(block_table, dtype=np.int64)
    if b < 0 or b >= bt.shape[0]:
        return np.zeros(0, np.int64), True
    j = np.arange(min(n, bt.shape[1] * page_size))
    blk = bt[b, j // page_size]
    ok = (blk >= 0) & (blk < num_blocks)
    return (blk * page_size + j % page_size)[ok], bool((~ok).any() or len(j) < n)


def attend_terms(q, k, v, scale: float):
    """out [H, dv] of q [H, dk] over keys k [n, dk] (or [H, n, dk]) and values v alike, and the
    terms of an error bound, all float64:

    * ``p`` [H, n]: the probabilities;  ``mass`` [H, dv]: sum_j p_j |v_j|;
    * ``qk`` [H]: max_j scale * sum_i |q_i k_ji|, the size of a score's terms;
    * ``smax`` [H]: max_j |s_j|.
    """
    H = q.shape[0]
    kh = k if k.ndim == 3 else k[None]
    vh = v if v.ndim == 3 else v[None]
    if kh.shape[1] == 0:
        z = np.zeros((H, vh.shape[2]))
        return z, dict(p=np.zeros((H, 0)), mass=z, qk=np.zeros(H), smax=np.zeros(H))
    s = np.matmul(kh, q[:, :, None])[:, :, 0] * scale
    e = np.exp(s - s.max(1, keepdims=True))
    p = e / e.sum(1, keepdims=True)
    out = np.matmul(p[:, None], vh)[:, 0]
    mass = np.matmul(p[:, None], np.abs(vh))[:, 0]
    qk = (np.matmul(np.abs(kh), np.abs(q)[:, :, None])[:, :, 0] * abs(scale)).max(1)
    return out, dict(p=p, mass=mass, qk=qk, smax=np.abs(s).max(1))


def decode(q_latent, q_rope, positions, seq_of_token, block_table, pool_rows, *, page_size: int,
           scale: float, fp8: bool, row_scale=None):
    """Absorbed latent attention, token by token: a list of (out [H, L], terms), and the error flag.
    q_latent [T, H, L], q_rope [T, H, R] float64.  The terms also hold ``row_scale`` and ``rows``
    of the entries attended to."""
    L, R = q_latent.shape[2], q_rope.shape[2]
    nb = pool_rows.shape[0]
    flat = pool_rows.reshape(nb * page_size, -1)
    res, error = [], False
    for t in range(len(positions)):
        b = 0 if seq_of_token is None else int(seq_of_token[t])
        at, bad = entries(b, max(0, int(positions[t]) + 1), block_table, nb, page_size)
        error |= bad
        sc = None if row_scale is None else np.asarray(row_scale)[at]
        x = row_values(flat[at], L, R, fp8=fp8, scale=sc)
        q = np.concatenate([q_latent[t], q_rope[t]], 1)
        out, terms = attend_terms(q, x, x[:, :L], scale)
        terms.update(rows=x, row_scale=sc)
        res.append((out, terms))
    return res, error


def prefill(q, k_nope, k_rope, v, cu_q, cu_k, *, scale: float, rows=None):
    """Expanded form, float64 arrays q [Tq, H, dk], k_nope [Tk, H, dn], k_rope [Tk, dr],
    v [Tk, H, dv]: {row: (out [H, dv], terms)} of the query rows asked for (None: all)."""
    res = {}
    H = q.shape[1]
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        for t in range(q0, q1):
            if rows is not None and t not in rows:
                continue
            n = max(0, (t - q0) + 1 + (k1 - k0) - (q1 - q0))
            kr = np.broadcast_to(k_rope[None, k0:k0 + n], (H, n, k_rope.shape[1]))
            k = np.concatenate([k_nope[k0:k0 + n].transpose(1, 0, 2), kr], 2)
            res[t] = attend_terms(q[t], k, v[k0:k0 + n].transpose(1, 0, 2), scale)
    return res
