"""Drafts that the tree decode rejects: every row that belongs to no accepted sequence keeps its bytes, and an
accepted one gives what it gives alone."""
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from test_gpu_latent import clean_error_word, dev  # noqa: F401
from test_gpu_latent_tree import Case

pytestmark = pytest.mark.gpu

CTX, CU = [40, 33, 20], [0, 3, 7, 12]
CASES = [  # bounds, contexts, accepted sequences
    (CU, CTX, [0, 1, 2]),
    ([0, 3, 2, 12], CTX, [0]),                   # decreasing; the last begins before the first ends
    ([0, 3, 7, 13], CTX, [0, 1]),                # past the last token
    ([-1, 3, 7, 12], CTX, [1, 2]),
    ([5, 3, 7, 12], CTX, [2]),                   # the second begins before a bound that was passed
    ([0, 3, 9, 12], CTX, [0, 1, 2]),             # other sizes
    ([0, 3, 9, 12], [40, -1, 20], [0, 2]),
    ([0, 4, 9, 11], [40, 1 << 30, 20], [0, 2]),
    ([0, 4, 9, 11], [(1 << 31) - 1, 33, -(1 << 31)], [1]),
    ([0, 20, 21, 22], CTX, []),
    ([3, 3, 3, 5], [0, 33, 20], [0, 1, 2]),      # (empty ones are accepted)
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [16, 20])
def test_rows_of_rejected_sequences_keep_their_bytes(dev, fp8, heads):  # noqa: F811
    c = Case(dev, CTX, [6, 6, 6], heads, fp8=fp8, seed=8)         # (entries of six drafted tokens each)
    i32 = dict(dtype=torch.int32, device=dev)
    ql, qr, pool, mask = c.args[0][:12], c.args[1][:12], c.args[2], c.args[5][:12].contiguous()
    for cu, ctx, good in CASES:
        out = torch.full((12, heads, 512), 9.0, dtype=torch.bfloat16, device=dev)
        c.fn()(ql, qr, pool, torch.tensor(ctx, **i32), torch.tensor(cu, **i32), mask, scale=c.scale, out=out)
        want = torch.full_like(out, 9.0)
        for b in good:
            alone = pool._replace(block_table=pool.block_table[b:b + 1].contiguous())
            c.fn()(ql, qr, alone, torch.tensor([ctx[b]], **i32), torch.tensor(cu[b:b + 2], **i32), mask, scale=c.scale,
                   out=want)
        code = spa.sparse_attn_paged_check_errors()
        assert code == (0 if len(good) == 3 else spa.SPA_STATUS["SPA_ERR_INDEX"]), (cu, ctx)
        lo, hi = [cu[b] for b in good], [cu[b + 1] for b in good]
        inside = torch.zeros(12, dtype=torch.bool)
        for x, y in zip(lo, hi):
            inside[x:y] = True
        assert bool((out[~inside.to(dev)] == 9.0).all()), (cu, ctx)
        assert bool(torch.isfinite(out[inside.to(dev)]).all())
        # (a sequence alone is shared out among the pairs of CTAs in another way: the parts' joining rounds differently)
        got, ref = out.double(), want.double()
        assert bool(((got - ref).abs() <= 2.0 ** -7 * ref.abs() + 2 * 2.0 ** -8 * 6.0).all()), (cu, ctx)
