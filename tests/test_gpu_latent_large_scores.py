"""Latent attention of drafted trees where scores are large: their maximum has to be held in 32 bits.

q's latent part is zero and its rotary part (A, 1, 0 ..), rows have rotary parts (r, d, 0 ..) of few bits, so that
a score A r + d is exact in the MMA (bf16) or off by two alignments of its fp32 sum (e4m3), and values are
whatever the latent parts hold.  What is left of the bounds of test_gpu_latent.py: no accumulation of products, no
rounding of q, and in place of 4 of the score's own roundings 10: two of 2^-23 in the sum, one each of a row's scale
into it, of the exponent's argument, of the reference and of a part's log-sum-exp, and of the merge's
difference of two of those (each 2^-24 of the largest score, the last two also between parts)."""
import numpy as np
import pytest
import torch

from oracle import latent_tree as otree
from test_gpu_latent import assert_within, clean_error_word, dev, f64, tolerance  # noqa: F401
from test_gpu_latent_tree import Case

pytestmark = pytest.mark.gpu


def large(dev, ctx, ns, H, fp8, base, grow, seed, L=128, page=64):
    """A case whose scores are A (base + 2 step) + d: A a number of -448 .. 448 a row of q, d in quarters below four;
    `grow`: steps along the sequence, so that the maximum moves at many tiles."""
    c = Case(dev, ctx, ns, H, L=L, R=16, page=page, fp8=fp8, seed=seed, scale=1.0)
    r = np.random.RandomState(seed)
    inp, T = c.inp, sum(ns)
    n = inp.rope.shape[0]
    inp.rope[:] = 0.0
    inp.rope[:, 0] = base
    if grow:
        at = inp.positions.float() / max(1, max(ctx))
        inp.rope[:, 0] = base + 2 * torch.floor(12 * at).to(torch.bfloat16)
    inp.rope[:, 1] = torch.from_numpy(r.randint(0, 16, n) / 4.0).to(torch.bfloat16)
    c.q[:] = 0.0
    a = r.randint(30, 113, (T, H)) * 4 * r.choice([-1, 1], (T, H))
    c.q[..., L] = torch.from_numpy(a).to(torch.bfloat16)
    c.q[..., L + 1] = 1.0
    c.pool, c.rows, c.row_scale = c.placed(dev)
    c.args = (c.q[..., :L].contiguous().to(dev), c.q[..., L:].contiguous().to(dev), c.pool) + c.args[3:]
    return c


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("grow", [False, True])
@pytest.mark.parametrize("base", [256, 274, 330])
@pytest.mark.parametrize("ctx,ns,H", [([90], [9], 16), ([40, 3], [24, 5], 20), ([3000, 50], [7, 12], 64),
                                      ([26000], [6], 16)])
def test_large_scores(dev, ctx, ns, H, base, grow, fp8):  # noqa: F811
    """Scores of 3e4 to 1.6e5 of both signs whose best entries differ by a few units: units of one tile, units cut
    between pairs of CTAs, and several tiles a pair."""
    c = large(dev, ctx, ns, H, fp8, base, grow, seed=base + H)
    out = f64(c.run())
    L = c.q.shape[2] - 16
    want = otree.tree_decode(f64(c.q[..., :L]), f64(c.q[..., L:]), c.ctx, c.cu, c.mask, c.inp.block_table.numpy(),
                             c.rows, page_size=c.inp.page_size, scale=c.scale, fp8=fp8, row_scale=c.row_scale)
    for t, (o, terms) in want.items():
        terms["smax"] = 2.5 * terms["smax"]              # (10 roundings of the score in place of 4)
        tol = tolerance(o, terms, 0, rows=terms["rows"], row_scale=terms["row_scale"] if fp8 else None, qmax=0.0,
                        scale=c.scale)
        assert_within(out[t], o, tol, (t, ctx, ns))
