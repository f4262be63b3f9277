"""Rotary positions, norms of heads and the appends on the GPU against the float64 oracle.

Bounds, per value (the oracle's y, the pair's size P = m (|a| + |b|) after the norm):

* bf16 output: ``2^-8 |y|``;
* rotation: the angle's fraction of a turn in fp32 (``2 pi 2^-32 + pi 2^-24`` radians), sine and cosine within
  2^-23, their product with m, two products and a sum (3 times 2^-24): below ``10 * 2^-24 P``;
* norm: D squares summed in fp32 in any order (``D 2^-24``, halved by the root), rsqrt within 2^-22, a
  division, an addition and two products: below ``(D / 2 + 9) 2^-24`` of the value;
* e4m3: in codes z = y / scale, half a step, ``max(2^-4 |z|, 2^-10)``; the scale and the quotient are within
  ``4 * 2^-24`` of theirs, besides what the values are off.  A second code leaves half its own step of that.
"""
import numpy as np
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from oracle import e4m3_to_f64
from oracle import latent as olat
from oracle import rotary as orot
from test_gpu_latent import clean_error_word, dev, f64  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def table_for(R, dev, interleaved=True, scale=1.0, **kw):
    return spa.sparse_attn_rotary_table(R, interleaved=interleaved, scale=scale, device=dev, **kw)


def far(T, seed):
    """Positions from 0 to the largest, negative ones among them."""
    p = np.random.RandomState(seed).randint(-1000, 1 << 20, T).astype(np.int32)
    p[:4] = [0, (1 << 31) - 1, -5, 1 << 30][:T]
    return torch.from_numpy(p)


def rope_slack(x, table, start, R, **kw):
    return 10 * U * abs(table.scale) * orot.pair_sizes(x, start=start, R=R, interleaved=table.interleaved)


def within(got, want, tol, what=""):
    err = np.abs(got - want)
    assert np.all(np.isfinite(got)), what
    assert np.all(err <= tol), (what, (err - tol).max(), err.max())


SHAPES = [  # T, H, D, R, start
    (1, 1, 8, 8, None), (3, 5, 64, 64, None), (17, 64, 512, 64, None), (2, 128, 192, 64, 128), (33, 7, 128, 32, 0),
    (5, 20, 128, 128, None), (9, 3, 256, 256, 0), (4, 9, 1024, 64, 480), (6, 2, 1024, 256, 768), (7, 10, 72, 40, 8),
    (300, 33, 64, 16, 24), (2, 3, 64, 0, None),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,D,R,start", SHAPES)
def test_rope(dev, T, H, D, R, start, interleaved, inverse):  # noqa: F811
    g = torch.Generator().manual_seed(T + H + D)
    x = torch.randn((T, H, D), generator=g).to(torch.bfloat16)
    pos, tab = far(T, D), table_for(R, dev, interleaved, 1.25 if inverse else 1.0)
    s = D - R if start is None else start
    out = spa.sparse_attn_rope(x.to(dev), pos.to(dev), tab, start=start, inverse=inverse)
    want = orot.rotate(f64(x), pos.tolist(), tab.turns.tolist(), start=s, interleaved=interleaved,
                       scale=tab.scale, inverse=inverse)
    within(f64(out), want, 2.0 ** -8 * np.abs(want) + rope_slack(f64(x), tab, s, R))
    keep = np.ones(D, bool)
    keep[s:s + R] = False
    assert np.array_equal(f64(out)[..., keep], f64(x)[..., keep])
    # in place, on a view with gaps: the same bits, and nothing else of the buffer touched
    buf = torch.full((T, H + 1, D + 16), 7.0, dtype=torch.bfloat16, device=dev)
    view = buf[:, :H, 8:8 + D]
    view.copy_(x)
    assert spa.sparse_attn_rope(view, pos.to(dev), tab, start=start, inverse=inverse, out=view) is view
    assert torch.equal(view, out)
    view.fill_(7.0)
    assert bool((buf == 7.0).all())


@pytest.mark.parametrize("dtype", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,D,R,start", SHAPES)
def test_norm_rope(dev, T, H, D, R, start, interleaved, dtype):  # noqa: F811
    g = torch.Generator().manual_seed(T * H + D)
    x = (5.0 * torch.randn((T, (H + 2) * D), generator=g)).to(torch.bfloat16)
    x[0, :D] = 0.0
    x[-1, D:2 * D] *= 1e-12
    q, k = x[:, :H * D].unflatten(1, (H, D)), x[:, H * D:].unflatten(1, (2, D))
    w = [None if dtype is None else (1 + torch.randn(D, generator=g)).to(dtype) for _ in range(2)]
    pos, tab = far(T, H), table_for(R, dev, interleaved)
    xd = x.to(dev)
    qd, kd = xd[:, :H * D].unflatten(1, (H, D)), xd[:, H * D:].unflatten(1, (2, D))
    eps = 1e-6
    outs = spa.sparse_attn_norm_rope(qd, kd, pos.to(dev), tab, q_weight=None if dtype is None else w[0].to(dev),
                                     k_weight=None if dtype is None else w[1].to(dev), eps=eps, start=start)
    s = D - R if start is None else start
    for name, rows, wt, out in (("q", q, w[0], outs[0]), ("k", k, w[1], outs[1])):
        y = orot.norm(f64(rows), None if wt is None else wt.double().numpy(), eps)
        want = orot.rotate(y, pos.tolist(), tab.turns.tolist(), start=s, interleaved=interleaved)
        size = np.maximum(np.abs(want), orot.pair_sizes(y, start=s, R=R, interleaved=interleaved))
        within(f64(out), want, 2.0 ** -8 * np.abs(want) + (D / 2 + 9) * U * size + rope_slack(y, tab, s, R), name)
    # q alone, in place, and without a rotation
    spa.sparse_attn_norm_rope(qd, None, pos.to(dev), tab, q_weight=None if dtype is None else w[0].to(dev), eps=eps,
                              start=start, q_out=qd)
    assert torch.equal(qd, outs[0])
    bare, none = spa.sparse_attn_norm_rope(kd, None, pos.to(dev), None, eps=eps)
    want = orot.norm(f64(k), None, eps)
    within(f64(bare), want, (2.0 ** -8 + (D / 2 + 9) * U) * np.abs(want))
    assert none is None


def test_far_positions_keep_their_angles(dev):  # noqa: F811
    """Next to the largest position neighbours differ by the frequency, as they do at 0."""
    tab = table_for(64, dev, scaling="yarn", factor=32.0)
    base = (1 << 31) - 9
    x = torch.zeros((8, 1, 64), dtype=torch.bfloat16)
    x[..., 0::2] = 1.0
    pos = torch.arange(base, base + 8, dtype=torch.int32)
    out = f64(spa.sparse_attn_rope(x.to(dev), pos.to(dev), tab))
    want = orot.rotate(f64(x), pos.tolist(), tab.turns.tolist(), start=0, interleaved=True, scale=tab.scale)
    within(out, want, 2.0 ** -8 * np.abs(want) + 10 * U * tab.scale)


def code_tolerance(y, scale, rel, twice=None):
    """What a code's value may be off y (see the module's text): `rel` is what y may be off already; `twice`:
    values (a mask) that have a second code."""
    z = np.abs(y) / scale
    half = np.maximum(2.0 ** -4 * z, 2.0 ** -10)
    if twice is not None:
        # (where the first code is one step off, the second one takes that up, but for e4m3's largest)
        half = np.where(twice, np.maximum(2.0 ** -4 * half * 1.01, 2.0 ** -10), half)
    return (half + (rel + 8 * U) * z) * scale * (1 + 8 * U)


def paged(dev, lens, page, D, fp8, seed):  # noqa: F811
    from workloads import latent_inputs
    inp = latent_inputs(lens, 64, 8, page, seed=seed)
    kv = torch.full((inp.num_blocks, page, 2, D), 0x5A, dtype=torch.uint8, device=dev) if fp8 else \
        torch.full((inp.num_blocks, page, 2, D), 3.25, dtype=torch.bfloat16, device=dev)
    scales = [torch.full((inp.num_blocks * page,), -7.0, device=dev) for _ in range(2)] if fp8 else [None, None]
    return inp, spa.PagedPool(kv, inp.block_table.to(dev), *scales)


def slots(inp, entries, sid):
    bt = inp.block_table.numpy().astype(np.int64)
    return bt[sid, entries // inp.page_size] * inp.page_size + entries % inp.page_size


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("lens,page,D,R,start", [
    ([1], 64, 512, 64, None), ([70, 3, 200], 24, 512, 64, None), ([33, 0, 9], 1, 64, 64, 0), ([50], 16, 128, 40, 8),
    ([5, 4], 64, 512, 256, 128), ([2000, 700], 64, 448, 0, None)])
def test_kv_append(dev, lens, page, D, R, start, interleaved, norm):  # noqa: F811
    T = sum(lens)
    g = torch.Generator().manual_seed(T + D)
    kv = (4.0 * torch.randn((T, 2 * D + 8), generator=g)).to(torch.bfloat16)
    if T > 5:
        kv[1] = 0.0
        kv[2, :D] *= 1e-30
        kv[3, :D] *= 1e-4
        kv[3, 7] = 900.0
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16) if norm else None
    tab = table_for(R, dev, interleaved, 1.5) if R else None
    pos = far(T, 3)
    eps = 1e-5 if norm else None
    kvd, s = kv.to(dev), D - R if start is None else start
    k, v = f64(kv[:, :D]), f64(kv[:, D:2 * D])
    y = orot.norm(k, w.double().numpy(), eps) if norm else k
    rel = (D / 2 + 9) * U if norm else 0.0
    want, size = y, np.abs(y)
    if R:
        want = orot.rotate(y, pos.tolist(), tab.turns.tolist(), start=s, interleaved=interleaved, scale=tab.scale)
        size = np.maximum(np.abs(want), 1.5 * orot.pair_sizes(y, start=s, R=R, interleaved=interleaved))
    for fp8 in (False, True):
        inp, pool = paged(dev, lens, page, D, fp8, 11)
        sid, ent = inp.seq_of_token.numpy(), inp.positions.numpy()
        before = pool.kv.clone()
        fn = spa.sparse_attn_paged_kv_append_fp8 if fp8 else spa.sparse_attn_paged_kv_append
        fn(kvd[:, :D], kvd[:, D:2 * D], pos.to(dev), pool, tab, weight=None if w is None else w.to(dev), eps=eps,
           start=start, entries=inp.positions.to(dev), seq_of_token=inp.seq_of_token.to(dev))
        at = slots(inp, ent, sid)
        rows = pool.kv.view(-1, 2, D)
        if not fp8:
            within(f64(rows[at, 0]), want, 2.0 ** -8 * np.abs(want) + (rel + 10 * U) * size)
            assert torch.equal(rows[at, 1].cpu(), kv[:, D:2 * D])
        else:
            ks = pool.k_scale.cpu().double().numpy()[at]
            amax = np.abs(want).max(1)
            unit = np.where(amax > 0, amax / 448.0, 1.0)
            off = (rel + 10 * U) * size.max(1) / np.maximum(amax, 1e-300)      # of the row's maximum
            assert np.all(np.abs(ks - unit) <= (off + 4 * U) * unit)
            got = e4m3_to_f64(rows[at, 0].cpu().numpy()) * ks[:, None]
            within(got, want, code_tolerance(want, ks[:, None], 0.0) + (rel + 10 * U) * size)
            # V as the K/V write has it
            _, other = paged(dev, lens, page, D, True, 11)
            spa.sparse_attn_paged_kv_write_fp8(kvd[:, :D].contiguous(), kvd[:, D:2 * D].contiguous(),
                                               inp.positions.to(dev), other, seq_of_token=inp.seq_of_token.to(dev))
            assert torch.equal(rows[at, 1], other.kv.view(-1, 2, D)[at, 1])
            assert torch.equal(pool.v_scale, other.v_scale)
        rest = np.setdiff1d(np.arange(before.shape[0] * page), at)
        assert torch.equal(rows[rest], before.view(-1, 2, D)[rest])
        if fp8:
            assert bool((pool.k_scale[torch.from_numpy(rest).to(dev)] == -7.0).all())


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("lens,page,L,R", [([1], 64, 512, 64), ([70, 3, 200], 24, 512, 64), ([33, 0, 9], 1, 64, 0),
                                           ([50, 60], 16, 192, 40), ([1500, 900], 64, 512, 8)])
def test_latent_append(dev, lens, page, L, R, interleaved, norm):  # noqa: F811
    from workloads import latent_inputs
    inp = latent_inputs(lens, L, R, page, seed=5)
    T = sum(lens)
    g = torch.Generator().manual_seed(T)
    x = (4.0 * torch.randn((T, L + R), generator=g)).to(torch.bfloat16)
    if T > 5:
        x[1] = 0.0
        x[2] *= 1e-30
        x[3, 5] = 900.0
    w = (1 + 0.3 * torch.randn(L, generator=g)) if norm else None
    tab = table_for(R, dev, interleaved, 1.5) if R else None
    pos = far(T, 3)
    eps = 1e-5 if norm else None
    c, r = f64(x[:, :L]), f64(x[:, L:])
    c2 = orot.norm(c, w.double().numpy(), eps) if norm else c
    r2 = orot.rotate(r, pos.tolist(), tab.turns.tolist(), start=0, interleaved=interleaved, scale=1.5) if R else r
    want = np.concatenate([c2, r2], 1)
    slack = np.concatenate([(L / 2 + 9) * U * np.abs(c2) * norm,
                            15 * U * orot.pair_sizes(r, start=0, R=R, interleaved=interleaved)], 1)
    xd = x.to(dev)
    for fp8 in (False, True):
        rows, scale = (None if t is None else t.to(dev) for t in inp.pool(fp8))
        pool = spa.LatentPool(rows, inp.block_table.to(dev), R, scale)
        fn = spa.sparse_attn_latent_append_fp8 if fp8 else spa.sparse_attn_latent_append
        before = rows.clone()
        fn(xd[:, :L], xd[:, L:] if R else None, pos.to(dev), pool, tab, weight=None if w is None else w.to(dev),
           eps=eps, entries=inp.positions.to(dev), seq_of_token=inp.seq_of_token.to(dev))
        at = slots(inp, inp.positions.numpy(), inp.seq_of_token.numpy())
        flat = rows.view(-1, rows.shape[2])
        if not fp8:
            within(f64(flat[at]), want, 2.0 ** -8 * np.abs(want) + slack)
        else:
            s = scale.cpu().double().numpy()[at]
            amax = np.abs(want).max(1)
            unit = np.where(amax > 0, amax / 448.0, 1.0)
            assert np.all(np.abs(s - unit) <= slack.max(1) / 448.0 * 1.001 + 4 * U * unit)
            got = olat.row_values(flat[at].cpu().numpy(), L, R, fp8=True, scale=s)
            twice = np.arange(L + R) >= L
            within(got, want, code_tolerance(want, s[:, None], 0.0, twice) + slack)
        rest = np.setdiff1d(np.arange(flat.shape[0]), at)
        assert torch.equal(flat[rest].view(torch.uint8), before.view(-1, rows.shape[2])[rest].view(torch.uint8))


def test_appends_skip_what_has_no_place(dev):  # noqa: F811
    """Bad entries, pages, blocks and sequences: skipped, flagged, the others written."""
    inp, pool = paged(dev, [40, 40], 16, 64, False, 2)
    bt = pool.block_table.clone()
    bt[1, 1] = -1
    bt[1, 2] = 1 << 20
    pool = pool._replace(block_table=bt)
    ent = torch.tensor([0, -1, 1 << 30, 5, 20, 40, 3, 3], dtype=torch.int32, device=dev)
    sid = torch.tensor([0, 0, 0, 1, 1, 1, 2, -1], dtype=torch.int32, device=dev)
    k = torch.ones((8, 64), dtype=torch.bfloat16, device=dev)
    before = pool.kv.clone()
    spa.sparse_attn_paged_kv_append(k, 2 * k, ent, pool, None, entries=ent, seq_of_token=sid)
    assert spa.sparse_attn_paged_check_errors() == spa.SPA_STATUS["SPA_ERR_INDEX"]
    at = [int(bt[0, 0]) * 16, int(bt[1, 0]) * 16 + 5]
    rows, old = pool.kv.view(-1, 2, 64), before.view(-1, 2, 64)
    assert bool((rows[at, 0] == 1).all()) and bool((rows[at, 1] == 2).all())
    rest = np.setdiff1d(np.arange(rows.shape[0]), at)
    assert torch.equal(rows[rest], old[rest])
    lat = spa.LatentPool(torch.zeros((4, 16, 64), dtype=torch.bfloat16, device=dev), bt[:, :1].contiguous() % 4, 0)
    spa.sparse_attn_latent_append(k, None, ent, lat, None, seq_of_token=sid)
    assert spa.sparse_attn_paged_check_errors() == spa.SPA_STATUS["SPA_ERR_INDEX"]
    assert int((lat.rows != 0).any(-1).sum()) == 2


def test_nothing_to_do(dev):  # noqa: F811
    tab = table_for(8, dev)
    none = torch.zeros(0, dtype=torch.int32, device=dev)
    x = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=dev)
    assert spa.sparse_attn_rope(x, none, tab).shape == (0, 4, 64)
    assert spa.sparse_attn_norm_rope(x, x[:, :1], none, tab)[1].shape == (0, 1, 64)
    _, pool = paged(dev, [3], 16, 64, False, 2)
    spa.sparse_attn_paged_kv_append(x[:, 0], x[:, 0], none, pool, tab)


def test_refusals(dev):  # noqa: F811
    tab = table_for(64, dev)
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device=dev)
    pos = torch.zeros(4, dtype=torch.int32, device=dev)
    for call in (lambda: spa.sparse_attn_rope(x.float(), pos, tab), lambda: spa.sparse_attn_rope(x, pos[:3], tab),
                 lambda: spa.sparse_attn_rope(x, pos.long(), tab), lambda: spa.sparse_attn_rope(x, pos.cpu(), tab),
                 lambda: spa.sparse_attn_rope(x, pos, tab._replace(turns=tab.turns.cpu())),
                 lambda: spa.sparse_attn_rope(x, pos, tab._replace(turns=tab.turns.float())),
                 lambda: spa.sparse_attn_rope(x, pos, tab, out=x[:, :1]),
                 lambda: spa.sparse_attn_norm_rope(x, x[:2], pos, tab),
                 lambda: spa.sparse_attn_norm_rope(x, None, pos, tab, q_weight=torch.ones(32, device=dev))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: spa.sparse_attn_rope(x, pos, tab, start=8), lambda: spa.sparse_attn_rope(x, pos, tab, start=-8),
                 lambda: spa.sparse_attn_norm_rope(x, None, pos, tab, eps=0.0),
                 lambda: spa.sparse_attn_rope(x, pos, tab._replace(scale=float("inf"))),
                 lambda: spa.sparse_attn_rope(x[..., 4:60], pos, table_for(8, dev)),
                 lambda: spa.sparse_attn_rope(x[..., :60], pos, table_for(8, dev))):
        with pytest.raises(spa.SpaError):
            call()


def test_captured_and_on_another_stream(dev):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn((50, 8, 128), generator=g, device=dev).to(torch.bfloat16)
    pos = torch.arange(50, dtype=torch.int32, device=dev)
    tab = table_for(64, dev)
    want = spa.sparse_attn_norm_rope(x, None, pos, tab)[0]
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        spa.sparse_attn_norm_rope(x, None, pos, tab, q_out=out)
        spa.sparse_attn_rope(out, pos, tab, inverse=True, out=out)
        spa.sparse_attn_rope(out, pos, tab, out=out)
    back = spa.sparse_attn_rope(spa.sparse_attn_rope(want, pos, tab, inverse=True), pos, tab)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, back)
    again = spa.sparse_attn_norm_rope(x, None, pos, tab, stream=side)[0]
    torch.cuda.synchronize()
    assert torch.equal(again, want)
