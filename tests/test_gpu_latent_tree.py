"""Latent attention of drafted trees on the GPU against the float64 oracle (bounds as in
test_gpu_latent.py: what a weight and a score may be off are the decode's), and the steps of a draft's check
run together."""
import numpy as np
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from oracle import latent_tree as otree
from test_gpu_latent import assert_within, clean_error_word, dev, f64, place, tolerance  # noqa: F401
from workloads import bf16_bits, latent_inputs

pytestmark = pytest.mark.gpu


def random_trees(ns, words, seed):
    """Masks of random trees, the bits past a tree's size set at random (they mean nothing)."""
    r = np.random.RandomState(seed)
    mask = np.zeros((sum(ns), words), dtype=np.uint32)
    row = 0
    for n in ns:
        for i in range(n):
            bits = 0
            parent = r.randint(-1, i) if i else -1
            if parent >= 0:
                bits = sum(int(w) << (32 * k) for k, w in enumerate(mask[row + parent])) % (1 << n)
            bits |= 1 << i
            bits |= int(r.randint(0, 1 << 30)) << n
            for k in range(words):
                mask[row + i, k] = (bits >> (32 * k)) & 0xFFFFFFFF
        row += n
    return mask


class Case:
    def __init__(self, dev, ctx, ns, H, L=512, R=64, page=64, fp8=False, words=None, chain=False, seed=0, qscale=1.0,
                 scale=None):
        self.ctx, self.ns, self.fp8, self.R = ctx, ns, fp8, R
        self.inp = latent_inputs([c + n for c, n in zip(ctx, ns)], L, R, page, seed=seed)
        self.pool, self.rows, self.row_scale = self.placed(dev)
        g = torch.Generator().manual_seed(seed + 1)
        T = sum(ns)
        self.q = (qscale * torch.randn((T, H, L + R), generator=g)).to(torch.bfloat16)
        self.scale = (128 + R) ** -0.5 if scale is None else scale
        self.cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        words = max(1, -(-max(ns + [1]) // 32)) if words is None else words
        self.mask = None if chain else random_trees(ns, words, seed)
        i32 = dict(dtype=torch.int32, device=dev)
        self.args = (self.q[..., :L].contiguous().to(dev), self.q[..., L:].contiguous().to(dev) if R else None, self.pool,
                     torch.tensor(ctx, **i32), torch.tensor(self.cu, **i32),
                     None if chain else torch.from_numpy(self.mask.view(np.int32)).to(dev))

    def placed(self, dev):
        pool, rows, scale, *_ = place(self.inp, self.fp8, dev)
        return pool, rows, scale

    def fn(self):
        return spa.sparse_attn_latent_tree_decode_fp8 if self.fp8 else spa.sparse_attn_latent_tree_decode

    def run(self, **kw):
        return self.fn()(*self.args, scale=self.scale, **kw)

    def check(self, out):
        L = self.q.shape[2] - self.R
        want = otree.tree_decode(f64(self.q[..., :L]), f64(self.q[..., L:]), self.ctx, self.cu, self.mask,
                                 self.inp.block_table.numpy(), self.rows, page_size=self.inp.page_size,
                                 scale=self.scale, fp8=self.fp8, row_scale=self.row_scale)
        got = f64(out)
        for t, (o, terms) in want.items():
            tol = tolerance(o, terms, L + self.R, rows=terms["rows"],
                            row_scale=terms["row_scale"] if self.fp8 else None,
                            qmax=np.abs(f64(self.q[t])).max(1) if self.fp8 else None, scale=self.scale)
            assert_within(got[t], o, tol, (t, self.ctx, self.ns))


SHAPES = [  # contexts, drafted, heads, L, R, page
    ([0], [1], 1, 512, 64, 64), ([1], [1], 16, 512, 64, 64), ([63], [1], 64, 512, 64, 64), ([64], [2], 64, 512, 64, 64),
    ([100], [8], 16, 512, 64, 64), ([4000], [7], 64, 512, 64, 64), ([300, 0, 17, 129], [5, 33, 1, 12], 20, 512, 64, 24),
    ([400, 600], [24, 3], 128, 512, 64, 128), ([200, 90], [130, 70], 8, 512, 64, 64), ([77, 5, 9], [4, 0, 9], 130, 512, 8, 1),
    ([130], [20], 7, 64, 0, 16), ([500, 3], [9, 40], 48, 448, 40, 64), ([129, 66], [31, 65], 24, 192, 16, 40),
    ([30000], [4], 16, 512, 64, 64), ([20] * 70, [1 + i % 3 for i in range(70)], 16, 128, 64, 32),
    ([257, 640, 12], [17, 2, 29], 64, 320, 64, 64),
    # several tiles and units a pair of CTAs: pages of seven, eight and 64 entries
    ([5000, 900, 3000], [17, 9, 60], 128, 64, 16, 7), ([9000, 40], [30, 25], 64, 128, 8, 1),
    ([5000, 900, 3000], [17, 9, 60], 128, 64, 16, 8), ([2500] * 9, [11] * 9, 128, 128, 64, 64),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctx,ns,H,L,R,page", SHAPES)
def test_trees(dev, ctx, ns, H, L, R, page, fp8):  # noqa: F811
    c = Case(dev, ctx, ns, H, L, R, page, fp8, seed=len(ctx) + H)
    c.check(c.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_chain_without_a_mask(dev, fp8):  # noqa: F811
    c = Case(dev, [70, 0, 300], [5, 40, 1], 20, fp8=fp8, chain=True, seed=9)
    c.check(c.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_masks_that_leave_nothing_or_have_too_few_words(dev, fp8):  # noqa: F811
    c = Case(dev, [0, 50, 0], [40, 70, 3], 16, fp8=fp8, words=1, seed=4)
    c.mask[[0, 7, 39]] = 0                  # without context: nothing to see
    c.mask[42] = 0                          # the context alone
    c.args = c.args[:5] + (torch.from_numpy(c.mask.view(np.int32)).to(dev),)
    out = c.run()
    c.check(out)
    assert bool((out[[0, 7, 39]] == 0).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_what_is_not_seen_does_not_enter(dev, fp8):  # noqa: F811
    """NaN and infinities in the rows of drafted tokens that a token does not see, behind the last
    sequence's last row, and on pages of nobody: the outputs of those who do not see them keep their bits,
    those who see a NaN become NaN."""
    c = Case(dev, [90, 40], [12, 30], 16, fp8=fp8, page=16, seed=6)
    c.mask[:, 0] &= np.uint32((1 << 30) - 1)
    c.args = c.args[:5] + (torch.from_numpy(c.mask.view(np.int32)).to(dev),)
    want = c.run()
    rows, bt = c.pool.rows, c.inp.block_table.numpy()
    used = np.zeros(rows.shape[0] * 16, bool)
    at = lambda b, j: int(bt[b, j // 16]) * 16 + j % 16  # noqa: E731
    for b, (n, k) in enumerate(zip(c.ctx, c.ns)):
        used[[at(b, j) for j in range(n + k)]] = True
    flat = rows.view(-1, rows.shape[2])
    nan = 0x7F if fp8 else float("nan")
    flat[torch.from_numpy(~used).to(flat.device)] = nan
    if fp8:
        c.pool.scale[torch.from_numpy(~used).to(flat.device)] = float("nan")
    assert torch.equal(c.run().view(torch.int16), want.view(torch.int16))
    # entry 90 + 5 is NaN, 40 + 20 has infinities of both signs (e4m3 has none: an infinite scale)
    flat[at(0, 95)] = nan
    if fp8:
        c.pool.scale[at(1, 60)] = float("inf")
    else:
        flat[at(1, 60), ::2] = float("inf")
        flat[at(1, 60), 1::2] = float("-inf")
    got = c.run()
    see = (c.mask[:12, 0] >> 5) & 1
    see = np.concatenate([see, (c.mask[12:, 0] >> 20) & 1]).astype(bool)
    keep = torch.from_numpy(~see).to(got.device)
    assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16))
    assert bool(torch.isnan(got[torch.from_numpy(np.flatnonzero(see[:12])).to(got.device)]).all())
    assert see[:12].any() and see[12:].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_of_no_sequence_and_bad_sequences_keep_their_bytes(dev, fp8):  # noqa: F811
    c = Case(dev, [40, 33, 20], [3, 4, 5], 16, fp8=fp8, seed=8)
    ql, qr, pool, ctx, cu, mask = c.args
    want = c.run()
    pad = lambda t: torch.cat([t[:1], t, t[-2:]])  # noqa: E731
    out = torch.full((15, 16, 512), 9.0, dtype=torch.bfloat16, device=dev)
    args = (pad(ql), pad(qr), pool, ctx, cu + 1, pad(mask))
    c.fn()(*args, scale=c.scale, out=out)
    assert torch.equal(out[1:13], want) and bool((out[[0, 13, 14]] == 9.0).all())
    for bad_cu, bad_ctx in (([0, 3, 2, 12], [40, 33, 20]), ([0, 3, 7, 13], [40, 33, 20]), ([-1, 3, 7, 12], [40, 33, 20]),
                            ([0, 3, 7, 12], [40, -1, 20]), ([0, 3, 7, 12], [40, 33, 1 << 30]),
                            ([5, 3, 7, 12], [40, 33, 20])):
        out.fill_(9.0)
        i32 = dict(dtype=torch.int32, device=dev)
        c.fn()(ql, qr, pool, torch.tensor(bad_ctx, **i32), torch.tensor(bad_cu, **i32), mask, scale=c.scale,
               out=out[:12])
        assert spa.sparse_attn_paged_check_errors() == spa.SPA_STATUS["SPA_ERR_INDEX"]
        top = 0
        for b in range(3):
            lo, hi = bad_cu[b], bad_cu[b + 1]
            good = lo >= top and lo <= hi <= 12 and 0 <= bad_ctx[b] < 1000
            top = max(top, lo)
            if good and (lo, hi) == (int(c.cu[b]), int(c.cu[b + 1])):
                assert torch.equal(out[lo:hi], want[lo:hi])
        assert bool((out[12:] == 9.0).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [64, 16])
def test_unmapped_pages_are_left_out_and_flagged(dev, fp8, page):  # noqa: F811
    c = Case(dev, [300, 40], [9, 5], 20, fp8=fp8, page=page, seed=12)
    bt = c.inp.block_table.clone()
    bt[0, 1] = -1
    bt[0, 3] = c.inp.num_blocks
    c.inp.block_table = bt
    c.args = c.args[:2] + (c.pool._replace(block_table=bt.to(dev)),) + c.args[3:]
    out = c.run()
    assert spa.sparse_attn_paged_check_errors() == spa.SPA_STATUS["SPA_ERR_INDEX"]
    c.check(out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
def test_scales(dev, fp8, scale):  # noqa: F811
    c = Case(dev, [200], [6], 20, fp8=fp8, seed=13, scale=scale)
    c.check(c.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_growing_maxima(dev, fp8):  # noqa: F811
    """Scores that grow along the sequence, so that the running maximum moves at every tile."""
    c = Case(dev, [1500], [10], 16, fp8=fp8, seed=14)
    inp = c.inp
    inp.latent[:] = (inp.latent.float() * torch.linspace(0.1, 4.0, inp.latent.shape[0])[:, None]).to(torch.bfloat16)
    c.pool, c.rows, c.row_scale = c.placed(dev)
    c.args = c.args[:2] + (c.pool,) + c.args[3:]
    c.check(c.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_strided_queries_and_given_memory(dev, fp8):  # noqa: F811
    c = Case(dev, [130, 70], [5, 9], 20, fp8=fp8, seed=15)
    want = c.run()
    x = torch.zeros((14, 22, 600), dtype=torch.bfloat16, device=dev)
    x[:, 1:21, 8:520], x[:, 1:21, 528:592] = c.args[0], c.args[1]
    n = spa.sparse_attn_latent_tree_decode_workspace_size(c.args[0], c.pool, 2, fp8=fp8)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=dev)
    out = torch.empty_like(want)
    got = c.fn()(x[:, 1:21, 8:520], x[:, 1:21, 528:592], *c.args[2:], scale=c.scale, out=out, workspace=ws)
    assert got is out and torch.equal(out, want)
    if n > 16:
        with pytest.raises(spa.SpaError):
            c.fn()(*c.args, scale=c.scale, workspace=ws[:n - 16])


@pytest.mark.parametrize("fp8", [False, True])
def test_again_bound_captured_and_on_another_stream(dev, fp8):  # noqa: F811
    c = Case(dev, [3000, 10, 700], [20, 3, 40], 32, fp8=fp8, seed=16)
    want = c.run()
    for _ in range(5):
        assert torch.equal(c.run(), want)
    call = spa.bind_latent_tree_decode(*c.args, scale=c.scale, fp8=fp8)
    call()
    assert torch.equal(call.out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = c.run(stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
        second = c.run(workspace=call.workspace)
    torch.cuda.synchronize()
    assert torch.equal(other, want)
    for _ in range(3):
        call.out.zero_()
        second.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(call.out, want) and torch.equal(second, want)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_draft_is_checked(dev, fp8):  # noqa: F811
    """Projections to logits' inputs as a serving step has them: queries normalised and rotated, prompt and
    draft appended (the draft's angles are its depths), the tree attended to; every path of the tree
    gives what a decode of that path alone gives, within both calls' bounds."""
    g = torch.Generator(device=dev).manual_seed(3)
    randn = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    L, R, H, page, ctx = 512, 64, 16, 16, 150
    parents = [-1, 0, 0, 1, 3, 2, -1, 6]
    n, i32 = len(parents), dict(dtype=torch.int32, device=dev)
    paths = [[i] for i in range(n)]
    for i, p in enumerate(parents):
        paths[i] = (paths[p] if p >= 0 else []) + [i]
    depth = torch.tensor([len(p) - 1 for p in paths], **i32)
    mask = torch.tensor([[sum(1 << j for j in p)] for p in paths], **i32)
    tab = spa.sparse_attn_rotary_table(R, scaling="yarn", factor=8.0, device=dev)
    w = (1 + 0.1 * torch.randn(L, generator=g, device=dev)).to(torch.bfloat16)
    prompt, draft = randn(ctx, L + R), randn(n, L + R)
    q = spa.sparse_attn_norm_rope(randn(n, H, L + R), None, ctx + depth, tab)[0]
    ql, qr = q[..., :L], q[..., L:]
    bt = torch.randperm(64, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(4, 16).to(dev)
    rows = torch.zeros((64, page, L + (2 * R if fp8 else R)), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
    pool = spa.LatentPool(rows, bt, R, torch.zeros(64 * page, device=dev) if fp8 else None)
    sfx = "_fp8" if fp8 else ""
    append, tree = getattr(spa, "sparse_attn_latent_append" + sfx), getattr(spa, "sparse_attn_latent_tree_decode" + sfx)
    decode = getattr(spa, "sparse_attn_latent_decode" + sfx)
    pos = torch.arange(ctx, **i32)
    for b in (0, 1):
        append(prompt[:, :L], prompt[:, L:], pos, pool, tab, weight=w, eps=1e-6, seq_of_token=torch.full_like(pos, b))
    append(draft[:, :L], draft[:, L:], ctx + depth, pool, tab, weight=w, eps=1e-6,
           entries=ctx + torch.arange(n, **i32))
    out = tree(ql, qr, pool, torch.tensor([ctx], **i32), torch.tensor([0, n], **i32), mask, scale=0.06)
    for i, path in enumerate(paths):
        k = torch.tensor(path, device=dev)
        at = ctx + torch.arange(len(path), **i32)
        append(draft[k, :L], draft[k, L:], at, pool, tab, weight=w, eps=1e-6, seq_of_token=torch.ones_like(at))
        want = decode(ql[i:i + 1], qr[i:i + 1], pool, at[-1:], scale=0.06, seq_of_token=torch.ones(1, **i32))
        # values are normalised rows times weights about 1: |out| <= A < 8.  Each call: output and weights 2^-8 A
        # (e4m3: 2^-11 of them), scores and sums far below
        a, b = f64(out[i:i + 1]), f64(want)
        assert np.all(np.abs(a - b) <= 2.0 ** -8 * (np.abs(a) + np.abs(b)) + 2 * 2.0 ** -8 * 8.0), i
    assert spa.sparse_attn_paged_check_errors() == 0


def test_refusals(dev):  # noqa: F811
    c = Case(dev, [20, 9], [3, 2], 16, seed=21)
    ql, qr, pool, ctx, cu, mask = c.args
    for args in ((ql.float(), qr, pool, ctx, cu, mask), (ql, None, pool, ctx, cu, mask), (ql, qr[:, :8], pool, ctx, cu, mask),
                 (ql, qr, pool, ctx.long(), cu, mask), (ql, qr, pool, ctx, cu[:2], mask), (ql, qr, pool, ctx.cpu(), cu, mask),
                 (ql, qr, pool, ctx, cu, mask[:3]), (ql, qr, pool, ctx, cu, mask.cpu()), (ql, qr, pool, ctx, cu, mask[:, 0]),
                 (ql, qr, pool, torch.cat([ctx, ctx]), torch.cat([cu, cu[-2:]]), mask)):
        with pytest.raises(ValueError):
            spa.sparse_attn_latent_tree_decode(*args, scale=0.1)
    with pytest.raises(spa.SpaError):
        spa.sparse_attn_latent_tree_decode(*c.args, scale=float("nan"))
    with pytest.raises(TypeError):
        spa.sparse_attn_latent_tree_decode_fp8(*c.args, scale=0.1)
    none = torch.zeros(1, dtype=torch.int32, device=dev)
    out = spa.sparse_attn_latent_tree_decode(ql[:0], qr[:0], pool, none[:0], none, scale=0.1)
    assert out.shape == (0, 16, 512)
