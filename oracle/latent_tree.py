"""Latent attention of drafted tokens behind their context in the cache.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain numpy, float64, from the definition;
shares no code with the CUDA library.

Token i of sequence b sees entries ``j < context`` and the entries ``context + i'`` of the drafted
tokens i' whose bit is set in its mask (without masks: i' <= i).
"""
import numpy as np

from .latent import attend_terms, row_values


def visible(ctx: int, n: int, i: int, mask) -> list:
    """Entries that token i sees, in order; mask: its 32-bit words, or None."""
    if mask is None:
        return list(range(ctx + i + 1))
    words = [int(w) & 0xFFFFFFFF for w in mask]
    return list(range(ctx)) + [ctx + k for k in range(min(n, 32 * len(words))) if words[k // 32] >> (k % 32) & 1]


def tree_decode(q_latent, q_rope, context_lens, cu_tokens, mask, block_table, pool_rows, *, page_size: int,
                scale: float, fp8: bool, row_scale=None) -> dict:
    """{token: (out [H, L], terms)} of every token of every sequence (see ``oracle.latent.decode``)."""
    L, R = q_latent.shape[2], q_rope.shape[2]
    nb = pool_rows.shape[0]
    flat = pool_rows.reshape(nb * page_size, -1)
    bt = np.asarray(block_table, dtype=np.int64)
    res = {}
    for b in range(len(context_lens)):
        t0, n, ctx = int(cu_tokens[b]), int(cu_tokens[b + 1]) - int(cu_tokens[b]), int(context_lens[b])
        for i in range(n):
            j = np.array(visible(ctx, n, i, None if mask is None else mask[t0 + i]), dtype=np.int64)
            blk = bt[b, j // page_size]
            ok = (blk >= 0) & (blk < nb)
            at = (blk * page_size + j % page_size)[ok]
            sc = None if row_scale is None else np.asarray(row_scale)[at]
            x = row_values(flat[at], L, R, fp8=fp8, scale=sc)
            q = np.concatenate([q_latent[t0 + i], q_rope[t0 + i]], 1)
            out, terms = attend_terms(q, x, x[:, :L], scale)
            terms.update(rows=x, row_scale=sc)
            res[t0 + i] = (out, terms)
    return res
