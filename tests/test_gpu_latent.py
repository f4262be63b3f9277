"""Latent attention on the GPU against the float64 oracle: the cache's write and read exactly, the
absorbed and the expanded form within bounds derived from their arithmetic, and all of them run
together as a serving step would.

Bounds of an attention output, per element (``A = sum_j p_j |v_j|``, from the oracle):

* the output's rounding to bf16: ``2^-8 |out|``;
* probabilities rounded to bf16 before the value product: ``2^-8 A``.  e4m3 pools: a weight
  ``w = p * scale`` enters as an e5m2 and an e4m3 term of ``u = w * 2^k`` where 2^k brings the
  largest weight to at least 2^5: u is rounded to f16 (``2^-11 u``), the first term leaves
  ``2^-3 u``, the second ``2^-4`` of that or half of e4m3's smallest step, and below 2^-17 nothing of u
  is left, so the error is at most
  ``2^-11 w + min(2^-3 w + 2^-17 2^-5 w_max, 2^-7 w + 2^-10 2^-5 w_max)``;
* a score's error d (absolute, natural units) changes every p by at most a factor ``e^(2d)``:
  ``(e^(2d) - 1) A``.  d = the accumulation of W products in fp32 (tensor cores may truncate where
  they align a group: ``W 2^-23`` of the terms' sum ``qk``) + the score times log2(e) in fp32 and
  the exponential's argument (``4 * 2^-24 * smax``) + ex2.approx (2^-22).  e4m3 pools: the query as
  two e4m3 terms leaves ``2^-17 max|q|`` an element in place of an exact one;
* the accumulation of n weighted values in fp32: ``n 2^-23 A``.
"""
import numpy as np
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from oracle import bf16_to_f64
from oracle import latent as olat
from workloads import bf16_bits, latent_inputs

pytestmark = pytest.mark.gpu

SENTINEL = 0x5A


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    if torch.cuda.is_available():
        assert spa.sparse_attn_paged_check_errors() == 0, "an error word was left behind"


def f64(t):
    return bf16_to_f64(bf16_bits(t.cpu().contiguous()))


def tolerance(out, terms, n_products, v=None, rows=None, row_scale=None, qmax=None, scale=None):
    """Element-wise bound [H, dv] (see the module's text); row_scale given: an e4m3 pool."""
    p, A = terms["p"], terms["mass"]
    d = n_products * 2.0 ** -23 * terms["qk"] + 4 * 2.0 ** -24 * terms["smax"] + 2.0 ** -22
    if row_scale is None:
        weights = 2.0 ** -8 * A
    else:
        if p.shape[1]:
            w = p * row_scale[None]
            wmax = w.max(1, keepdims=True)
            werr = 2.0 ** -11 * w + np.minimum(2.0 ** -3 * w + 2.0 ** -22 * wmax,
                                               2.0 ** -7 * w + 2.0 ** -15 * wmax)
            codes = np.abs(rows[:, :out.shape[1]]) / row_scale[:, None]
            weights = werr @ codes
            d = d + abs(scale) * 2.0 ** -17 * qmax * np.abs(rows).sum(1).max()
        else:
            weights = 0.0
    n = p.shape[1]
    return 2.0 ** -8 * np.abs(out) + weights + ((np.exp(2 * d) - 1)[:, None] + n * 2.0 ** -23) * A \
        + 1e-30


def assert_within(got, out, tol, what):
    err = np.abs(got - out)
    assert np.all(np.isfinite(got)), what
    worst = (err - tol).max() if err.size else 0.0
    assert np.all(err <= tol), (what, "over the bound by", worst, "max error", err.max())


# ---- write and read -------------------------------------------------------------------------
def awkward(inp):
    """A few rows that are hard on the quantiser: zeros, signed zeros, one large element among tiny
    ones, half-way points, a tiny row (a scale below the reciprocal path's range)."""
    if inp.latent.shape[0] < 6:
        return inp
    L = inp.latent.shape[1]
    inp.latent[0] = 0.0
    inp.rope[0] = -0.0
    inp.latent[1] = -0.0
    inp.latent[2] *= 1e-4
    inp.latent[2, 5] = 1000.0
    inp.latent[3] = torch.tensor([((8 + (i % 8)) + 0.5) * 2.0 ** (-(i % 6)) for i in range(L)])
    inp.latent[3, 0] = 448.0
    inp.latent[4] *= 1e-30
    inp.rope[4] *= 1e-30
    return inp


def place(inp, fp8, dev, sentinel=False, **kw):
    """The pool on the GPU and the oracle's copy after both wrote the rows."""
    rows, scale = inp.pool(fp8)
    if sentinel:
        rows.view(torch.uint8).fill_(SENTINEL)
        if fp8:
            scale.fill_(-7.0)
    o_rows = (rows.numpy() if fp8 else bf16_bits(rows)).copy()
    o_scale = scale.numpy().copy() if fp8 else None
    dropped = olat.write(bf16_bits(inp.latent), bf16_bits(inp.rope), inp.positions.numpy(),
                         inp.seq_of_token.numpy(), inp.block_table.numpy(), o_rows,
                         page_size=inp.page_size, scale=o_scale, fp8=fp8)
    pool = spa.LatentPool(rows.to(dev), inp.block_table.to(dev), inp.rope.shape[1],
                          scale.to(dev) if fp8 else None)
    f = spa.sparse_attn_latent_write_fp8 if fp8 else spa.sparse_attn_latent_write
    rope = inp.rope.to(dev) if inp.rope.shape[1] else None
    f(inp.latent.to(dev), rope, inp.positions.to(dev), pool, seq_of_token=inp.seq_of_token.to(dev), **kw)
    return pool, o_rows, o_scale, dropped


CACHE_CASES = {
    "one": dict(lens=[1], L=512, R=64, ps=64),
    "ragged": dict(lens=[300, 1, 77], L=512, R=64, ps=64),
    "p24": dict(lens=[130, 50], L=512, R=64, ps=24),
    "p1": dict(lens=[9, 8], L=64, R=8, ps=1),
    "norope": dict(lens=[40, 3], L=128, R=0, ps=16),
    "odd": dict(lens=[33, 65], L=448, R=40, ps=7),
    "many": dict(lens=[12000], L=64, R=16, ps=128),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", sorted(CACHE_CASES))
def test_write_and_read_exact(dev, case, fp8):
    c = CACHE_CASES[case]
    inp = awkward(latent_inputs(c["lens"], c["L"], c["R"], c["ps"], seed=5))
    pool, o_rows, o_scale, dropped = place(inp, fp8, dev, sentinel=True)
    assert not dropped
    assert np.array_equal(pool.rows.view(torch.uint8).cpu().numpy(),
                          o_rows.view(np.uint8).reshape(*o_rows.shape[:2], -1))
    if fp8:
        assert np.array_equal(pool.scale.cpu().numpy().view(np.uint32), o_scale.view(np.uint32))
    # the read, in another order and with repeats
    order = np.random.default_rng(6).integers(0, len(inp.positions), len(inp.positions))
    pos, sid = inp.positions[order], inp.seq_of_token[order]
    f = spa.sparse_attn_latent_read_fp8 if fp8 else spa.sparse_attn_latent_read
    got = f(pos.to(dev), pool, seq_of_token=sid.to(dev)).cpu()
    if not fp8:
        want = torch.cat([inp.latent, inp.rope], 1)[order]
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        return
    at = np.array([int(inp.block_table[b, x // c["ps"]]) * c["ps"] + x % c["ps"]
                   for b, x in zip(sid.tolist(), pos.tolist())])
    flat, L = torch.from_numpy(o_rows.reshape(-1, o_rows.shape[2])[at]), c["L"]
    v = flat.view(torch.float8_e4m3fn).float()       # fp32 products, as the definition says
    x = torch.cat([v[:, :L], v[:, L:L + c["R"]] + v[:, L + c["R"]:]], 1)
    want = (x * torch.from_numpy(o_scale[at])[:, None]).to(torch.bfloat16)
    assert torch.equal(got.float(), want.float())


@pytest.mark.parametrize("fp8", [False, True])
def test_write_and_read_of_what_does_not_exist(dev, fp8):
    inp = latent_inputs([70, 30], 128, 16, 8, seed=7)
    inp.block_table[0, 2] = -1                       # entries 16 .. 23 unmapped
    inp.block_table[0, 5] = inp.num_blocks           # entries 40 .. 47 outside the pool
    inp.positions[3] = -1
    inp.positions[60] = 8 * inp.block_table.shape[1]  # past the table
    inp.seq_of_token[71] = 2
    inp.seq_of_token[72] = -1
    pool, o_rows, o_scale, dropped = place(inp, fp8, dev, sentinel=True)
    assert dropped and spa.sparse_attn_paged_check_errors() == spa.SPA_STATUS["SPA_ERR_INDEX"]
    assert np.array_equal(pool.rows.view(torch.uint8).cpu().numpy(),
                          o_rows.view(np.uint8).reshape(*o_rows.shape[:2], -1))
    f = spa.sparse_attn_latent_read_fp8 if fp8 else spa.sparse_attn_latent_read
    got = f(inp.positions.to(dev), pool, seq_of_token=inp.seq_of_token.to(dev)).cpu()
    assert spa.sparse_attn_paged_check_errors() == spa.SPA_STATUS["SPA_ERR_INDEX"]
    gone = [t for t in range(100) if t in (3, 60, 71, 72) or 16 <= t < 24 or 40 <= t < 48]
    assert not got[gone].view(torch.int16).any()
    kept = [t for t in range(100) if t not in gone]
    if not fp8:
        want = torch.cat([inp.latent, inp.rope], 1)
        assert torch.equal(got[kept].view(torch.int16), want[kept].view(torch.int16))
    assert got[kept].float().abs().amax(1).min() > 0


@pytest.mark.parametrize("fp8", [False, True])
def test_write_and_read_strided(dev, fp8):
    """latent and rope as the two parts of one projection's output, out as part of a wider buffer,
    the pool a view into a larger allocation, an explicit stream."""
    inp = latent_inputs([50, 21], 192, 32, 16, seed=8)
    both = torch.zeros((71, 240), dtype=torch.bfloat16, device=dev)
    both[:, :192], both[:, 200:232] = inp.latent.to(dev), inp.rope.to(dev)
    rows, scale = inp.pool(fp8)
    big = torch.full((rows.numel() + 4096,), SENTINEL, dtype=rows.dtype, device=dev) if fp8 else \
        torch.zeros(rows.numel() + 4096, dtype=rows.dtype, device=dev)
    view = big[1024:1024 + rows.numel()].view(rows.shape)
    view.copy_(rows)
    pool = spa.LatentPool(view, inp.block_table.to(dev), 32, scale.to(dev) if fp8 else None)
    kw = dict(seq_of_token=inp.seq_of_token.to(dev))
    pos = inp.positions.to(dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    wide = torch.full((71, 256), 7.0, dtype=torch.bfloat16, device=dev)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        (spa.sparse_attn_latent_write_fp8 if fp8 else spa.sparse_attn_latent_write)(
            both[:, :192], both[:, 200:232], pos, pool, **kw)
    (spa.sparse_attn_latent_read_fp8 if fp8 else spa.sparse_attn_latent_read)(
        pos, pool, out=wide[:, 16:240], stream=s, **kw)
    s.synchronize()
    got = wide[:, 16:240].float().cpu()
    x = torch.cat([inp.latent, inp.rope], 1).float()
    assert bool((wide[:, :16] == 7).all()) and bool((wide[:, 240:] == 7).all())
    if fp8:   # half a step of e4m3, and of its smallest step at the row's scale
        step = x.abs().amax(1, keepdim=True) / 448 * 2.0 ** -10
        assert bool(((got - x).abs() <= (2.0 ** -4 + 2.0 ** -8) * x.abs() + step).all())
    else:
        assert torch.equal(got, x)


def test_one_row_written_twice_keeps_the_others(dev):
    """A step that writes a batch's next rows leaves every earlier row as it was."""
    inp = latent_inputs([40], 64, 16, 16, seed=9)
    pool, o_rows, _, _ = place(inp, True, dev)
    before = pool.rows.clone()
    new = torch.randn((1, 64), device=dev).to(torch.bfloat16)
    spa.sparse_attn_latent_write_fp8(new, torch.zeros((1, 16), dtype=torch.bfloat16, device=dev),
                                     torch.tensor([17], dtype=torch.int32, device=dev), pool)
    at = int(inp.block_table[0, 1]) * 16 + 1
    same = (pool.rows == before).view(-1, 96).all(1).cpu()
    assert not same[at] and same.sum() == len(same) - 1


# ---- absorbed form --------------------------------------------------------------------------
def decode_case(dev, lens, H, L, R, ps, fp8, q=1, seed=0, scale=None, big=1.0, mutate=None,
                positions=None, q_pad=0):
    """Runs the decode of the last q tokens of every sequence and checks it; returns what it made."""
    inp = latent_inputs(lens, L, R, ps, seed=seed)
    pool, o_rows, o_scale, _ = place(inp, fp8, dev)
    sid = torch.tensor([b for b in range(len(lens)) for _ in range(q)], dtype=torch.int32)
    pos = torch.tensor([n - q + i for n in lens for i in range(q)], dtype=torch.int32) \
        if positions is None else torch.tensor(positions, dtype=torch.int32)
    g = torch.Generator().manual_seed(seed + 100)
    T = len(pos)
    ql = (big * torch.randn((T, H, L + q_pad), generator=g)).to(torch.bfloat16)[..., :L]
    qr = (big * torch.randn((T, H, R + q_pad), generator=g)).to(torch.bfloat16)[..., :R]
    scale = (L + R) ** -0.5 if scale is None else scale
    if mutate is not None:
        mutate(pool, inp, sid)
        o_rows = pool.rows.cpu().numpy() if fp8 else bf16_bits(pool.rows.cpu())
        o_scale = pool.scale.cpu().numpy() if fp8 else None
    f = spa.sparse_attn_latent_decode_fp8 if fp8 else spa.sparse_attn_latent_decode
    out = f(ql.to(dev), qr.to(dev) if R else None, pool, pos.to(dev), scale=scale,
            seq_of_token=sid.to(dev))
    err = spa.sparse_attn_paged_check_errors()
    got = out.float().cpu().numpy().astype(np.float64)
    want, bad = olat.decode(f64(ql), f64(qr), pos.numpy(), sid.numpy(), inp.block_table, o_rows,
                            page_size=ps, scale=scale, fp8=fp8, row_scale=o_scale)
    assert err == (spa.SPA_STATUS["SPA_ERR_INDEX"] if bad else 0)
    for t, (o, terms) in enumerate(want):
        qmax = max(np.abs(f64(ql[t])).max(), np.abs(f64(qr[t])).max() if R else 0.0)
        tol = tolerance(o, terms, L + R + (R if fp8 else 0), rows=terms["rows"],
                        row_scale=terms["row_scale"], qmax=qmax, scale=scale)
        assert_within(got[t], o, tol, ("token", t, "position", int(pos[t])))
    return pool, ql, qr, pos, sid, out


DECODE_CASES = {
    "one_entry": dict(lens=[1], H=64, L=512, R=64, ps=64),
    "tile_edges": dict(lens=[63, 64, 65, 127, 128, 129], H=64, L=512, R=64, ps=64),
    "ragged_h128": dict(lens=[700, 3, 190, 1], H=128, L=512, R=64, ps=64),
    "h16_p24": dict(lens=[301, 24, 25], H=16, L=512, R=64, ps=24),
    "h1": dict(lens=[500], H=1, L=512, R=64, ps=32),
    "h20_p100": dict(lens=[450, 99], H=20, L=512, R=64, ps=100),
    "h130": dict(lens=[129, 66], H=130, L=512, R=64, ps=128),
    "l64_norope_p3": dict(lens=[200, 5], H=65, L=64, R=0, ps=3),
    "l448_r40_p1": dict(lens=[150], H=32, L=448, R=40, ps=1),
    "l128_r8_p16": dict(lens=[333, 17], H=64, L=128, R=8, ps=16),
    "l192_r64_p2": dict(lens=[131], H=64, L=192, R=64, ps=2),
    "l192_p64": dict(lens=[200, 64], H=64, L=192, R=64, ps=64),
    "l64_norope_p64": dict(lens=[130, 7], H=20, L=64, R=0, ps=64),
    "l320_r8_p128": dict(lens=[300], H=64, L=320, R=8, ps=128),
    "l384_r24_p192": dict(lens=[450, 191, 193], H=64, L=384, R=24, ps=192),
    "q3": dict(lens=[260, 66, 3], H=64, L=512, R=64, ps=64, q=3),
    "long": dict(lens=[9000], H=64, L=512, R=64, ps=64),
    "many_tokens": dict(lens=[5 + 7 * i for i in range(170)], H=8, L=64, R=16, ps=16),
    "strided_q": dict(lens=[90, 200], H=24, L=256, R=32, ps=32, q_pad=24),
    "sharp": dict(lens=[400, 130], H=64, L=512, R=64, ps=64, big=8.0),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", sorted(DECODE_CASES))
def test_decode_against_oracle(dev, case, fp8):
    decode_case(dev, fp8=fp8, seed=len(case), **DECODE_CASES[case])


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_positions_inside_and_before_the_sequence(dev, fp8):
    """Queries of one call at any position of their sequences: none, the first, the middle."""
    pool, *_, out = decode_case(dev, [300, 140], 64, 512, 64, 64, fp8, q=4, seed=31,
                                positions=[-1, 0, 100, 299, 139, 64, -1, 63])
    assert not out[0].any() and not out[6].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_leaves_out_what_does_not_exist(dev, fp8):
    """Unmapped and bad pages in the middle, a whole sequence unmapped, a bad sequence id: the rest
    is attended to, and NaN in every row that is not (the pools start as NaN) stays out."""
    def mutate(pool, inp, sid):
        bt = pool.block_table
        bt[0, 1] = -1
        bt[0, 4] = inp.num_blocks + 3
        bt[1, :] = -1
        inp.block_table[:] = bt.cpu()
        sid[5] = 6                                   # (there are sequences 0 .. 5)
        sid[4] = -2
    *_, out = decode_case(dev, [500, 80, 33, 64, 10, 12], 64, 512, 64, 32, fp8, seed=32,
                          mutate=mutate)
    assert not out[1].any() and not out[4].any() and not out[5].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_past_the_block_table(dev, fp8):
    """A position past the table's last page attends to the entries there are."""
    decode_case(dev, [112, 64], 32, 128, 16, 16, fp8, seed=33, positions=[2000000000, 70])


def test_decode_scores_of_any_size(dev):
    """Scores far past exp's range in either direction (the maximum is taken out first), and a
    scale of zero and below zero."""
    decode_case(dev, [200, 70], 16, 128, 16, 16, False, seed=34, big=30.0, scale=5.0)
    decode_case(dev, [200, 70], 16, 128, 16, 16, False, seed=35, scale=0.0)
    decode_case(dev, [200, 70], 16, 128, 16, 16, True, seed=36, scale=-0.1)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[70], [4000]])
def test_decode_query_that_is_not_finite(dev, lens, fp8):
    """NaN or infinity in one head's query makes that head's output NaN and leaves the others alone."""
    inp = latent_inputs(lens, 512, 64, 64, seed=31)
    pool, _, _, _ = place(inp, fp8, dev)
    g = torch.Generator().manual_seed(131)
    ql = torch.randn((1, 70, 512), generator=g).to(torch.bfloat16).to(dev)
    qr = torch.randn((1, 70, 64), generator=g).to(torch.bfloat16).to(dev)
    pos = torch.tensor([lens[0] - 1], dtype=torch.int32, device=dev)
    f = spa.sparse_attn_latent_decode_fp8 if fp8 else spa.sparse_attn_latent_decode
    want = f(ql, qr, pool, pos, scale=0.04)
    assert torch.isfinite(want).all()
    ql[0, 3, 100] = float("nan")
    ql[0, 66, 511] = float("inf")
    qr[0, 40, 5] = float("-inf")
    got = f(ql, qr, pool, pos, scale=0.04)
    gone = torch.tensor([3, 40, 66], device=dev)
    assert torch.isnan(got[0, gone]).all()
    rest = torch.ones(70, dtype=torch.bool, device=dev)
    rest[gone] = False
    assert torch.equal(got[0, rest], want[0, rest])
    assert spa.sparse_attn_paged_check_errors() == 0


def test_decode_rows_of_very_different_scales(dev):
    """e4m3 rows whose scales differ by factors of 2^40."""
    def mutate(pool, inp, sid):
        bt = pool.block_table[0].long()
        at = (bt[:, None] * 16 + torch.arange(16, device=dev)).reshape(-1)
        pool.scale[at[::3]] *= 2.0 ** -40
    decode_case(dev, [150], 16, 128, 16, 16, True, seed=37, mutate=mutate, scale=1e-3)


def test_decode_a_sink_and_a_long_tail(dev):
    """One entry with most of the weight and thousands with very little each: the tail counts."""
    for fp8 in (False, True):
        inp = latent_inputs([6000], 64, 0, 64, seed=38)
        inp.latent[:] = 0.0
        inp.latent[:, 0] = -1.0                      # the tail: value 1 in channel 1
        inp.latent[:, 1] = 1.0
        inp.latent[5, 0], inp.latent[5, 1] = 1.0, 0.0
        pool, o_rows, o_scale, _ = place(inp, fp8, dev)
        q = torch.zeros((1, 8, 64), dtype=torch.bfloat16)
        q[..., 0] = torch.arange(1, 9) * 0.75        # weights of the tail e^-1.5 .. e^-12 of the sink's
        f = spa.sparse_attn_latent_decode_fp8 if fp8 else spa.sparse_attn_latent_decode
        pos = torch.tensor([5999], dtype=torch.int32)
        out = f(q.to(dev), None, pool, pos.to(dev), scale=1.0)
        want, _ = olat.decode(f64(q), np.zeros((1, 8, 0)), pos.numpy(), None, inp.block_table, o_rows,
                              page_size=64, scale=1.0, fp8=fp8, row_scale=o_scale)
        o, terms = want[0]
        tol = tolerance(o, terms, 64, rows=terms["rows"], row_scale=terms["row_scale"], qmax=6.0,
                        scale=1.0)
        assert_within(f64(out[0]), o, tol, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_deterministic_and_workspace_contents_free(dev, fp8):
    """The same call twice gives the same bits, whatever the workspace held, and the workspace is
    no larger than the size asked for."""
    pool, ql, qr, pos, sid, out = decode_case(dev, [3000, 50], 64, 512, 64, 64, fp8, seed=39)
    n = spa.sparse_attn_latent_decode_workspace_size(ql, pool, pos, fp8=fp8)
    f = spa.sparse_attn_latent_decode_fp8 if fp8 else spa.sparse_attn_latent_decode
    for fill in (0x00, 0xFF, 0x7F):
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device=dev)
        again = f(ql.to(dev), qr.to(dev), pool, pos.to(dev), scale=576 ** -0.5,
                  seq_of_token=sid.to(dev), workspace=ws[:max(n, 16)])
        assert torch.equal(again.view(torch.int16), out.view(torch.int16))
        assert bool((ws[max(n, 16):] == fill).all())
    if n > 0:
        with pytest.raises(spa.SpaError) as e:
            f(ql.to(dev), qr.to(dev), pool, pos.to(dev), scale=1.0, seq_of_token=sid.to(dev),
              workspace=ws[:n - 16])
        assert e.value.status == spa.SPA_STATUS["SPA_ERR_WORKSPACE"]


def test_decode_graphs_that_share_a_workspace(dev):
    """Two captured decodes of different batches with one workspace, launched in turn."""
    a = decode_case(dev, [2000, 30], 64, 512, 64, 64, False, seed=40)
    b = decode_case(dev, [65, 900, 700], 128, 512, 64, 32, True, seed=41)
    calls = []
    n = max(spa.sparse_attn_latent_decode_workspace_size(x[1], x[0], x[3], fp8=f)
            for x, f in ((a, False), (b, True)))
    ws = torch.zeros(max(n, 16), dtype=torch.uint8, device=dev)
    for (pool, ql, qr, pos, sid, _), fp8 in ((a, False), (b, True)):
        calls.append(spa.bind_latent_decode(ql.to(dev), qr.to(dev), pool, pos.to(dev), fp8=fp8,
                                            scale=576 ** -0.5, seq_of_token=sid.to(dev),
                                            workspace=ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for c in calls:
        with torch.cuda.stream(side):
            c()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    for _ in range(3):
        for c, x, g in zip(calls, (a, b), graphs):
            c.out.zero_()
            g.replay()
            assert torch.equal(c.out.view(torch.int16), x[5].view(torch.int16))


def test_decode_on_two_streams_at_once(dev):
    a = decode_case(dev, [2500, 300], 64, 512, 64, 64, False, seed=42)
    pool, ql, qr, pos, sid, out = a
    args = (ql.to(dev), qr.to(dev), pool, pos.to(dev))
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = [spa.bind_latent_decode(*args, scale=576 ** -0.5, seq_of_token=sid.to(dev), stream=s)
             for s in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for c in calls:
            c()
    torch.cuda.synchronize()
    for c in calls:
        assert torch.equal(c.out.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_chain_without_synchronisation(dev, fp8):
    """Write and decode step after step on one stream, q and the new rows in buffers that the next step
    overwrites, one workspace: every step's output is that of the same call made alone afterwards."""
    start, steps, H = 300, 40, 64
    inp = latent_inputs([start + steps, 77], 512, 64, 64, seed=33)
    rows, scale = inp.pool(fp8)
    pool = spa.LatentPool(rows.to(dev), inp.block_table.to(dev), 64, scale.to(dev) if fp8 else None)
    write = spa.sparse_attn_latent_write_fp8 if fp8 else spa.sparse_attn_latent_write
    decode = spa.sparse_attn_latent_decode_fp8 if fp8 else spa.sparse_attn_latent_decode
    x, r = inp.latent.to(dev), inp.rope.to(dev)
    keep = torch.ones(len(x), dtype=torch.bool)
    keep[start:start + steps] = False
    keep = keep.to(dev)
    write(x[keep], r[keep], inp.positions.to(dev)[keep], pool, seq_of_token=inp.seq_of_token.to(dev)[keep])
    g = torch.Generator().manual_seed(133)
    qs = torch.randn((steps, 2, H, 576), generator=g).to(torch.bfloat16).to(dev)
    pos = torch.tensor([[start + i, 76] for i in range(steps)], dtype=torch.int32, device=dev)
    sid = torch.tensor([0, 1], dtype=torch.int32, device=dev)
    q, p, row, rope = qs[0].clone(), pos[0].clone(), x[:1].clone(), r[:1].clone()
    n = spa.sparse_attn_latent_decode_workspace_size(q[..., :512], pool, p, fp8=fp8)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    outs = torch.empty((steps, 2, H, 512), dtype=torch.bfloat16, device=dev)
    torch.cuda.synchronize()
    for i in range(steps):
        row.copy_(x[start + i:start + i + 1])
        rope.copy_(r[start + i:start + i + 1])
        p.copy_(pos[i])
        q.copy_(qs[i])
        write(row, rope, p[:1], pool)
        decode(q[..., :512], q[..., 512:], pool, p, scale=0.04, seq_of_token=sid, workspace=ws, out=outs[i])
    torch.cuda.synchronize()
    for i in range(steps):
        alone = decode(qs[i][..., :512], qs[i][..., 512:], pool, pos[i], scale=0.04, seq_of_token=sid)
        torch.cuda.synchronize()
        assert torch.equal(outs[i], alone), i
    assert torch.isfinite(outs).all() and spa.sparse_attn_paged_check_errors() == 0


def test_decode_and_cache_past_4_gigabytes(dev):
    """Rows whose byte offsets pass 2^32: pages at the end of a large pool."""
    ps, nb = 64, 64000                               # 64000 * 64 rows of 1152 bytes: 4.7 GB
    inp = latent_inputs([200, 100], 512, 64, ps, seed=43)
    inp.block_table[inp.block_table >= 0] += nb - inp.num_blocks
    rows = torch.empty((nb, ps, 576), dtype=torch.bfloat16, device=dev)
    pool = spa.LatentPool(rows, inp.block_table.to(dev), 64)
    sid, pos = inp.seq_of_token.to(dev), inp.positions.to(dev)
    spa.sparse_attn_latent_write(inp.latent.to(dev), inp.rope.to(dev), pos, pool, seq_of_token=sid)
    got = spa.sparse_attn_latent_read(pos, pool, seq_of_token=sid).cpu()
    x = torch.cat([inp.latent, inp.rope], 1)
    assert torch.equal(got, x)
    q = torch.randn((2, 64, 576), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    out = spa.sparse_attn_latent_decode(q[..., :512].to(dev), q[..., 512:].to(dev), pool,
                                        torch.tensor([199, 99], dtype=torch.int32, device=dev),
                                        scale=0.05, seq_of_token=torch.tensor([0, 1], dtype=torch.int32, device=dev))
    for t, (lo, hi) in enumerate([(0, 200), (200, 300)]):
        o, terms = olat.attend_terms(f64(q[t]), f64(x[lo:hi]), f64(x[lo:hi, :512]), 0.05)
        assert_within(f64(out[t]), o, tolerance(o, terms, 576), t)


# ---- expanded form --------------------------------------------------------------------------
def prefill_case(dev, nq, nk, H, dn, dr, dv, seed=0, rows=None, big=1.0, scale=None, mutate=None,
                 gap=0):
    g = torch.Generator().manual_seed(seed)
    cu_q = np.concatenate([[0], np.cumsum(nq)]) + gap
    cu_k = np.concatenate([[0], np.cumsum(nk)]) + gap
    Tq, Tk = int(cu_q[-1]) + gap, int(cu_k[-1]) + gap
    q = (big * torch.randn((Tq, H, dn + dr), generator=g)).to(torch.bfloat16)
    kv = torch.randn((Tk, H, dn + dv), generator=g).to(torch.bfloat16)
    kr = torch.randn((Tk, dr), generator=g).to(torch.bfloat16)
    if mutate is not None:
        mutate(q, kv, kr)
    scale = (dn + dr) ** -0.5 if scale is None else scale
    kv_d = kv.to(dev)
    out = torch.full((Tq, H, dv), -77.0, dtype=torch.bfloat16, device=dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    res = spa.sparse_attn_latent_prefill(q.to(dev), kv_d[..., :dn], kr.to(dev) if dr else None,
                                         kv_d[..., dn:], i32(cu_q), i32(cu_k), scale=scale, out=out)
    assert res is out and spa.sparse_attn_paged_check_errors() == 0
    want = olat.prefill(f64(q), f64(kv[..., :dn]), f64(kr), f64(kv[..., dn:]), cu_q, cu_k,
                        scale=scale, rows=rows)
    got = f64(out)
    for t, (o, terms) in want.items():
        assert_within(got[t], o, tolerance(o, terms, dn + dr), ("row", t))
    inside = np.zeros(Tq, bool)
    inside[cu_q[0]:cu_q[-1]] = True
    assert np.all(got[~inside] == -77.0)             # rows of no sequence keep their bytes
    return got


PREFILL_CASES = {
    "one": dict(nq=[1], nk=[1], H=16, dn=128, dr=64, dv=128),
    "edges": dict(nq=[127, 128, 129], nk=[127, 128, 129], H=4, dn=128, dr=64, dv=128),
    "ragged": dict(nq=[1, 300, 7, 64], nk=[1, 300, 7, 64], H=4, dn=128, dr=64, dv=128),
    "chunk": dict(nq=[100, 1, 33], nk=[700, 513, 33], H=4, dn=128, dr=64, dv=128),
    "decode_like": dict(nq=[1, 1, 1], nk=[300, 2, 129], H=20, dn=128, dr=64, dv=128),
    "empty_sequences": dict(nq=[0, 5, 0, 3], nk=[4, 9, 0, 3], H=3, dn=128, dr=64, dv=128),
    "more_queries_than_keys": dict(nq=[200, 9], nk=[30, 0], H=2, dn=128, dr=64, dv=128),
    "norope": dict(nq=[150, 40], nk=[150, 90], H=3, dn=128, dr=0, dv=128),
    "narrow": dict(nq=[90, 131], nk=[90, 200], H=5, dn=40, dr=24, dv=72),
    "tiny_widths": dict(nq=[70], nk=[140], H=2, dn=8, dr=8, dv=8),
    "dv64": dict(nq=[140], nk=[300], H=2, dn=64, dr=32, dv=64),
    "gap": dict(nq=[50, 60], nk=[70, 80], H=2, dn=128, dr=64, dv=128, gap=13),
    "sharp": dict(nq=[260], nk=[390], H=2, dn=128, dr=64, dv=128, big=12.0),
    "two_tiles_and_more": dict(nq=[520], nk=[777], H=2, dn=128, dr=64, dv=128),
}


@pytest.mark.parametrize("case", sorted(PREFILL_CASES))
def test_prefill_against_oracle(dev, case):
    prefill_case(dev, seed=len(case), **PREFILL_CASES[case])


def test_prefill_long_at_some_rows(dev):
    rows = {0, 1, 255, 256, 1000, 2047, 2999}
    prefill_case(dev, [3000], [3000], 8, 128, 64, 128, seed=51, rows=rows)
    prefill_case(dev, [400], [5000], 8, 128, 64, 128, seed=52, rows={0, 127, 128, 399})


def test_prefill_items_by_halves(dev):
    """Six items of 256 queries a head, a few more than the device has SMs: those of the second round are
    taken by single tiles of 128 queries.  (One sequence's last item has no second tile.)"""
    H = (torch.cuda.get_device_properties(dev).multi_processor_count + 20) // 6 + 1
    prefill_case(dev, [300, 77, 700], [333, 77, 700], H, 32, 16, 32, seed=53,
                 rows={0, 127, 128, 255, 256, 299, 300, 376, 377, 633, 1076})


def test_prefill_many_sequences(dev):
    """More sequences than a warp has lanes, several times over, some of them empty."""
    nq = [(7 * i) % 40 if i % 5 else 0 for i in range(100)]
    nq[70] = 300
    nk = [n + (11 * i) % 50 for i, n in enumerate(nq)]
    prefill_case(dev, nq, nk, 3, 32, 16, 32, seed=59)


@pytest.mark.parametrize("scale", [-0.07, 0.0])
def test_prefill_negative_and_zero_scale(dev, scale):
    prefill_case(dev, [200, 30], [200, 170], 2, 128, 64, 128, seed=58, scale=scale)


def test_prefill_other_sequences_stay_out(dev):
    """NaN in every row of the sequences before and after, and behind the last one."""
    def mutate(q, kv, kr):
        for x in (kv, kr):
            x[:40] = float("nan")
            x[40 + 133:] = float("nan")
    g = torch.Generator().manual_seed(53)
    nq, nk, H = [20, 133, 50], [40, 133, 50], 3
    q = torch.randn((203, H, 192), generator=g).to(torch.bfloat16)
    kv = torch.randn((260, H, 256), generator=g).to(torch.bfloat16)
    kr = torch.randn((260, 64), generator=g).to(torch.bfloat16)
    mutate(q, kv, kr)
    cu_q, cu_k = [0, 20, 153, 203], [0, 40, 173, 223]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    kv_d = kv.to(dev)
    out = spa.sparse_attn_latent_prefill(q.to(dev), kv_d[..., :128], kr.to(dev), kv_d[..., 128:],
                                         i32(cu_q), i32(cu_k), scale=0.07)
    want = olat.prefill(f64(q), f64(kv[..., :128]), f64(kr), f64(kv[..., 128:]), cu_q, cu_k,
                        scale=0.07, rows=set(range(20, 153)))
    got = f64(out)
    for t, (o, terms) in want.items():
        assert_within(got[t], o, tolerance(o, terms, 192), t)


def test_prefill_masked_keys_of_any_size_stay_out(dev):
    """Keys that are NaN, infinite or of the type's lowest value reach no query before them."""
    for value in (float("nan"), float("inf"), -3.38e38):
        def mutate(q, kv, kr):
            kv[100:, :, :128] = value
            kr[100:] = value
        prefill_case(dev, [180], [180], 2, 128, 64, 128, seed=54, rows=set(range(100)),
                     mutate=mutate)


def test_prefill_bad_bounds_are_left_out(dev):
    """A sequence whose bounds run backwards or past the rows is skipped and flagged; the others
    are computed."""
    H = 2
    g = torch.Generator().manual_seed(55)
    q = torch.randn((60, H, 192), generator=g).to(torch.bfloat16)
    kv = torch.randn((60, H, 256), generator=g).to(torch.bfloat16)
    kr = torch.randn((60, 64), generator=g).to(torch.bfloat16)
    kv_d = kv.to(dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    for cu_q, cu_k, good in (([0, 20, 40, 61], [0, 20, 40, 60], (0, 1)),
                             ([0, 20, 10, 60], [0, 20, 40, 60], (0,)),
                             ([0, 20, 40, 60], [0, 20, 61, 60], (0,)),
                             ([-1, 20, 40, 60], [0, 20, 40, 60], (1, 2)),
                             ([0, 20, 40, 60], [0, -5, 40, 60], (2,))):
        out = torch.full((60, H, 128), -77.0, dtype=torch.bfloat16, device=dev)
        spa.sparse_attn_latent_prefill(q.to(dev), kv_d[..., :128], kr.to(dev), kv_d[..., 128:],
                                       i32(cu_q), i32(cu_k), scale=0.07, out=out)
        assert spa.sparse_attn_paged_check_errors() == spa.SPA_STATUS["SPA_ERR_INDEX"]
        got = f64(out)
        for b in good:
            nq, nk = [cu_q[b], cu_q[b + 1]], [cu_k[b], cu_k[b + 1]]
            want = olat.prefill(f64(q), f64(kv[..., :128]), f64(kr), f64(kv[..., 128:]), nq, nk,
                                scale=0.07)
            for t, (o, terms) in want.items():
                assert_within(got[t], o, tolerance(o, terms, 192), (cu_q, t))
        owned = {t for b in good for t in range(cu_q[b], cu_q[b + 1])}
        if cu_q == [0, 20, 40, 61]:
            assert np.all(got[40:] == -77.0)


def test_prefill_strided_inputs_and_streams(dev):
    """Head-major storage and padded rows, on another stream, captured and replayed."""
    H, T = 3, 150
    g = torch.Generator().manual_seed(56)
    q = torch.randn((H, T, 200), generator=g).to(torch.bfloat16)
    k = torch.randn((H, T, 136), generator=g).to(torch.bfloat16)
    v = torch.randn((T, H + 1, 128), generator=g).to(torch.bfloat16)
    kr = torch.randn((T, 72), generator=g).to(torch.bfloat16)
    qd, kd, vd, rd = (x.to(dev) for x in (q, k, v, kr))
    views = (qd.transpose(0, 1)[..., :192], kd.transpose(0, 1)[..., 8:], rd[:, :64], vd[:, 1:])
    cu = torch.tensor([0, 100, T], dtype=torch.int32, device=dev)
    out = torch.zeros((T, H, 128), dtype=torch.bfloat16, device=dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    spa.sparse_attn_latent_prefill(*views, cu, cu, scale=0.07, out=out, stream=s)
    s.synchronize()
    want = olat.prefill(f64(q).transpose(1, 0, 2)[..., :192], f64(k).transpose(1, 0, 2)[..., 8:],
                        f64(kr)[:, :64], f64(v)[:, 1:], [0, 100, T], [0, 100, T], scale=0.07)
    got = f64(out)
    for t, (o, terms) in want.items():
        assert_within(got[t], o, tolerance(o, terms, 192), t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spa.sparse_attn_latent_prefill(*views, cu, cu, scale=0.07, out=out)
    out.zero_()
    for _ in range(2):
        graph.replay()
    assert np.array_equal(f64(out), got)


# ---- together -------------------------------------------------------------------------------
@pytest.mark.parametrize("fp8", [False, True])
def test_a_serving_run(dev, fp8):
    """A prompt in two chunks, then decoding steps: the rows are written, the second chunk's prefix
    is read back and up-projected for the expanded form, and every decoded token's absorbed output,
    up-projected, agrees with the expanded form of the whole sequence.  Both forms see the same
    cached rows, so they differ by their roundings alone: each output within its own bound of the
    float64 value."""
    L, R, H, dn, dv, ps, n = 128, 32, 4, 64, 64, 16, 150
    inp = latent_inputs([n], L, R, ps, seed=61)
    rows, scale = inp.pool(fp8)
    pool = spa.LatentPool(rows.to(dev), inp.block_table.to(dev), R, scale.to(dev) if fp8 else None)
    write = spa.sparse_attn_latent_write_fp8 if fp8 else spa.sparse_attn_latent_write
    read = spa.sparse_attn_latent_read_fp8 if fp8 else spa.sparse_attn_latent_read
    decode = spa.sparse_attn_latent_decode_fp8 if fp8 else spa.sparse_attn_latent_decode
    g = torch.Generator().manual_seed(62)
    w_uk = (torch.randn((H, dn, L), generator=g) / 8).to(torch.bfloat16)
    w_uv = (torch.randn((H, dv, L), generator=g) / 8).to(torch.bfloat16)
    q = torch.randn((n, H, dn + R), generator=g).to(torch.bfloat16)
    c, r, pos = inp.latent.to(dev), inp.rope.to(dev), inp.positions.to(dev)
    s = (dn + R) ** -0.5
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    outs = torch.zeros((n, H, dv), dtype=torch.bfloat16, device=dev)
    keys = {}
    for lo, hi in ((0, 70), (70, 140)):
        write(c[lo:hi], r[lo:hi], pos[lo:hi], pool)
        x = read(pos[:hi], pool)                     # the prefix and the chunk, as cached
        k = torch.einsum("tl,hdl->thd", x[:, :L].float(), w_uk.to(dev).float()).to(torch.bfloat16)
        v = torch.einsum("tl,hdl->thd", x[:, :L].float(), w_uv.to(dev).float()).to(torch.bfloat16)
        outs[lo:hi] = spa.sparse_attn_latent_prefill(q[lo:hi].to(dev), k, x[:, L:], v,
                                                     i32([0, hi - lo]), i32([0, hi]), scale=s)
        keys[hi] = (f64(k), f64(x[:, L:]), f64(v))
    for hi, (k, kr, v) in keys.items():
        want = olat.prefill(f64(q[hi - 70:hi]), k, kr, v, [0, 70], [0, hi], scale=s)
        for t, (o, terms) in want.items():
            assert_within(f64(outs[hi - 70 + t]), o, tolerance(o, terms, dn + R), (hi, t))
    absorbed = []
    for t in range(140, n):
        write(c[t:t + 1], r[t:t + 1], pos[t:t + 1], pool)
        ql = torch.einsum("hd,hdl->hl", q[t, :, :dn].double(), w_uk.double()).to(torch.bfloat16)
        absorbed.append((ql, decode(ql[None].to(dev), q[t:t + 1, :, dn:].to(dev), pool, pos[t:t + 1],
                                    scale=s)))
    flat = pool.rows.cpu().numpy() if fp8 else bf16_bits(pool.rows.cpu())
    sc = pool.scale.cpu().numpy() if fp8 else None
    for t, (ql, out) in zip(range(140, n), absorbed):
        want, _ = olat.decode(f64(ql)[None], f64(q[t:t + 1, :, dn:]), [t], None, inp.block_table, flat,
                              page_size=ps, scale=s, fp8=fp8, row_scale=sc)
        o, terms = want[0]
        tol = tolerance(o, terms, L + 2 * R, rows=terms["rows"], row_scale=terms["row_scale"],
                        qmax=float(ql.abs().max().clamp_min(q[t].abs().max())), scale=s)
        assert_within(f64(out[0]), o, tol, t)


def test_refused_devices_and_shapes(dev):
    inp = latent_inputs([20], 64, 16, 16, seed=63)
    pool, *_ = place(inp, False, dev)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device=dev)
    qr = torch.zeros((1, 4, 16), dtype=torch.bfloat16, device=dev)
    pos = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        spa.sparse_attn_latent_decode(q, qr, pool, pos, scale=1.0)
    with pytest.raises(ValueError, match="unit last stride"):
        spa.sparse_attn_latent_decode(q.expand(1, 4, 64).transpose(1, 2), qr, pool, pos.to(dev), scale=1.0)
    with pytest.raises(spa.SpaError) as e:           # rows that are not 16-byte aligned
        flat = torch.zeros(4 * 66 + 2, dtype=torch.bfloat16, device=dev)
        spa.sparse_attn_latent_decode(flat[2:].view(1, 4, 66)[..., :64], qr, pool, pos.to(dev), scale=1.0)
    assert e.value.status == spa.SPA_STATUS["SPA_ERR_ALIGN"]
