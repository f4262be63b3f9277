"""Latent attention: what the entry points refuse on the host, before touching a GPU (CPU only)."""
import ctypes
import os

import pytest
import torch

import sparse_paged_attention_gb300 as spa
from sparse_paged_attention_gb300 import SpaLatentPoolC, SpaLatentPrefillC, SpaLatentProblemC

S = spa.SPA_STATUS


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses: host validation is tested without a GPU")
    if not os.path.exists(spa.library_path()):
        from sparse_paged_attention_gb300.build import build_library
        build_library()
    return spa.load_library()


def pool(**kw):
    f = dict(rows=0x10000, scale=0x20000, block_table=0x30000, num_blocks=64, page_size=64,
             bt_stride=8, latent_dim=512, rope_dim=64)
    f.update(kw)
    return SpaLatentPoolC(*[f[n] for n, _ in SpaLatentPoolC._fields_])


BAD_POOLS = [
    (dict(rows=None), "SPA_ERR_NULL"), (dict(block_table=None), "SPA_ERR_NULL"),
    (dict(rows=0x10008), "SPA_ERR_ALIGN"), (dict(latent_dim=0), "SPA_ERR_SHAPE"),
    (dict(latent_dim=96), "SPA_ERR_UNSUPPORTED"), (dict(latent_dim=576), "SPA_ERR_UNSUPPORTED"),
    (dict(rope_dim=-8), "SPA_ERR_SHAPE"), (dict(rope_dim=12), "SPA_ERR_UNSUPPORTED"),
    (dict(rope_dim=72), "SPA_ERR_UNSUPPORTED"), (dict(num_blocks=0), "SPA_ERR_SHAPE"),
    (dict(page_size=0), "SPA_ERR_SHAPE"), (dict(bt_stride=0), "SPA_ERR_SHAPE"),
    (dict(num_blocks=1 << 25), "SPA_ERR_UNSUPPORTED"),
]


def write(lib, p, fp8=False, latent=0x40000, ls=512, rope=0x50000, rs=64, T=5, pos=0x60000, B=1):
    f = lib.sparse_attn_latent_write_fp8 if fp8 else lib.sparse_attn_latent_write
    return f(latent, ls, rope, rs, T, pos, None, B, None if p is None else ctypes.byref(p), None)


def read(lib, p, fp8=False, n=5, pos=0x60000, B=1, out=0x70000, os_=576):
    f = lib.sparse_attn_latent_read_fp8 if fp8 else lib.sparse_attn_latent_read
    return f(None if p is None else ctypes.byref(p), n, pos, None, B, out, os_, None)


def problem(**kw):
    f = dict(num_tokens=4, num_seqs=2, num_heads=64, scale=0.07, positions=0x60000,
             seq_of_token=None, q_latent=0x80000, q_rope=0x90000, q_latent_stride_t=64 * 512,
             q_latent_stride_h=512, q_rope_stride_t=64 * 64, q_rope_stride_h=64)
    f.update(kw)
    return SpaLatentProblemC(*[f[n] for n, _ in SpaLatentProblemC._fields_])


def decode(lib, p, pr, fp8=False, out=0xA0000, ws=0xB0000, wb=1 << 40):
    f = lib.sparse_attn_latent_decode_fp8 if fp8 else lib.sparse_attn_latent_decode
    return f(None if p is None else ctypes.byref(p), None if pr is None else ctypes.byref(pr), out,
             ws, wb, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad,code", BAD_POOLS)
def test_bad_pools_are_refused_by_every_entry_point(lib, bad, code, fp8):
    p = pool(**bad)
    assert write(lib, p, fp8) == S[code]
    assert read(lib, p, fp8) == S[code]
    assert decode(lib, p, problem(), fp8) == S[code]


def test_e4m3_pools_need_scales(lib):
    p = pool(scale=None)
    assert write(lib, p, True) == read(lib, p, True) == decode(lib, p, problem(), True) == \
        S["SPA_ERR_NULL"]


def test_write_and_read_refusals(lib):
    p = pool()
    assert write(lib, None) == read(lib, None) == S["SPA_ERR_NULL"]
    assert write(lib, p, T=-1) == read(lib, p, n=-1) == S["SPA_ERR_SHAPE"]
    assert write(lib, p, B=0) == read(lib, p, B=0) == S["SPA_ERR_SHAPE"]
    assert write(lib, p, ls=-8) == write(lib, p, rs=-8) == read(lib, p, os_=-8) == S["SPA_ERR_SHAPE"]
    assert read(lib, p, os_=568) == S["SPA_ERR_SHAPE"]
    assert write(lib, p, T=0) == read(lib, p, n=0) == S["SPA_OK"]
    for bad in (dict(latent=None), dict(rope=None), dict(pos=None)):
        assert write(lib, p, **bad) == S["SPA_ERR_NULL"]
    for bad in (dict(latent=0x40002), dict(rope=0x50008), dict(ls=516), dict(rs=68)):
        assert write(lib, p, **bad) == S["SPA_ERR_ALIGN"]
    assert read(lib, p, out=None) == read(lib, p, pos=None) == S["SPA_ERR_NULL"]
    assert read(lib, p, out=0x70008) == read(lib, p, os_=580) == S["SPA_ERR_ALIGN"]
    # without a rotary part its pointer is not looked at; the call then stops at the device query
    assert write(lib, pool(rope_dim=0), rope=None, rs=0) == S["SPA_ERR_CUDA"]
    assert write(lib, p) == read(lib, p) == S["SPA_ERR_CUDA"]


def test_decode_refusals(lib):
    p = pool()
    assert decode(lib, None, problem()) == decode(lib, p, None) == S["SPA_ERR_NULL"]
    for bad in (dict(num_tokens=-1), dict(num_seqs=0), dict(num_heads=0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(q_latent_stride_t=-8), dict(q_rope_stride_h=-8),
                dict(q_latent_stride_h=504), dict(q_latent_stride_t=0), dict(q_rope_stride_t=56)):
        assert decode(lib, p, problem(**bad)) == S["SPA_ERR_SHAPE"]
    assert decode(lib, p, problem(num_tokens=1 << 20, num_heads=1 << 12)) == S["SPA_ERR_UNSUPPORTED"]
    assert decode(lib, p, problem(num_tokens=0)) == S["SPA_OK"]
    for bad in (dict(positions=None), dict(q_latent=None), dict(q_rope=None)):
        assert decode(lib, p, problem(**bad)) == S["SPA_ERR_NULL"]
    assert decode(lib, p, problem(), out=None) == S["SPA_ERR_NULL"]
    for bad in (dict(q_latent=0x80008), dict(q_rope=0x90002), dict(q_latent_stride_t=64 * 512 + 4),
                dict(q_latent_stride_h=516), dict(q_rope_stride_t=68), dict(q_rope_stride_h=68)):
        assert decode(lib, p, problem(**bad)) == S["SPA_ERR_ALIGN"]
    assert decode(lib, p, problem(), out=0xA0008) == S["SPA_ERR_ALIGN"]
    assert decode(lib, p, problem()) == S["SPA_ERR_CUDA"]
    assert lib.sparse_attn_latent_decode_workspace_size(None, ctypes.byref(p)) == 0
    assert lib.sparse_attn_latent_decode_workspace_size(ctypes.byref(problem()), None) == 0


def prefill(lib, out=0xA0000, **kw):
    f = dict(num_q=10, num_k=20, num_seqs=2, num_heads=4, nope_dim=128, rope_dim=64, v_dim=128,
             scale=0.07, q=0x10000, k_nope=0x20000, k_rope=0x30000, v=0x40000, q_stride_t=768,
             q_stride_h=192, k_nope_stride_t=1024, k_nope_stride_h=256, k_rope_stride_t=64,
             v_stride_t=1024, v_stride_h=256, cu_q=0x50000, cu_k=0x60000)
    f.update(kw)
    p = SpaLatentPrefillC(*[f[n] for n, _ in SpaLatentPrefillC._fields_])
    return lib.sparse_attn_latent_prefill(ctypes.byref(p), out, None)


def test_prefill_refusals(lib):
    assert lib.sparse_attn_latent_prefill(None, 0xA0000, None) == S["SPA_ERR_NULL"]
    for bad in (dict(num_q=-1), dict(num_k=-1), dict(num_seqs=-1), dict(num_heads=0),
                dict(nope_dim=0), dict(v_dim=0), dict(rope_dim=-8), dict(scale=float("nan")),
                dict(q_stride_t=-8), dict(q_stride_t=184), dict(q_stride_h=184),
                dict(k_nope_stride_h=120), dict(k_nope_stride_t=0), dict(k_rope_stride_t=56),
                dict(v_stride_h=120), dict(v_stride_t=120),
                dict(v_stride_t=1 << 39)):
        assert prefill(lib, **bad) == S["SPA_ERR_SHAPE"], bad
    for bad in (dict(nope_dim=132), dict(nope_dim=136), dict(v_dim=4), dict(v_dim=136),
                dict(rope_dim=4), dict(rope_dim=72), dict(num_q=1 << 20, num_heads=1 << 12)):
        assert prefill(lib, **bad) == S["SPA_ERR_UNSUPPORTED"], bad
    for bad in (dict(q=None), dict(k_nope=None), dict(k_rope=None), dict(v=None), dict(cu_q=None),
                dict(cu_k=None), dict(out=None)):
        assert prefill(lib, **bad) == S["SPA_ERR_NULL"], bad
    for bad in (dict(q=0x10008), dict(k_nope=0x20002), dict(k_rope=0x30004), dict(v=0x40008),
                dict(q_stride_t=772), dict(v_stride_h=260), dict(k_rope_stride_t=68),
                dict(out=0xA0008)):
        assert prefill(lib, **bad) == S["SPA_ERR_ALIGN"], bad
    assert prefill(lib, num_q=0) == prefill(lib, num_seqs=0) == S["SPA_OK"]
    # no keys at all: key and value pointers are not looked at
    assert prefill(lib, num_k=0, k_nope=None, k_rope=None, v=None) == S["SPA_ERR_CUDA"]
    assert prefill(lib) == S["SPA_ERR_CUDA"]


def test_python_refusals_before_the_library():
    t = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)   # CPU tensors: refused at the latest
    p = spa.LatentPool(t(4, 8, 80), torch.zeros((1, 4), dtype=torch.int32), 16)
    pos = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        spa.sparse_attn_latent_write_fp8(t(3, 64), t(3, 16), pos, p)
    with pytest.raises(ValueError, match="scale"):
        spa.sparse_attn_latent_read_fp8(pos, spa.LatentPool(t(4, 8, 96, dt=torch.uint8),
                                                           p.block_table, 16))
    with pytest.raises(ValueError, match="latent"):
        spa.sparse_attn_latent_write(t(3, 72), t(3, 16), pos, p)
    with pytest.raises(ValueError, match="rope"):
        spa.sparse_attn_latent_write(t(3, 64), None, pos, p)
    with pytest.raises(ValueError, match="same number"):
        spa.sparse_attn_latent_write(t(3, 64), t(2, 16), pos, p)
    with pytest.raises(ValueError, match="positions"):
        spa.sparse_attn_latent_write(t(3, 64), t(3, 16), pos.long(), p)
    with pytest.raises(ValueError, match="CUDA"):
        spa.sparse_attn_latent_write(t(3, 64), t(3, 16), pos, p)
    with pytest.raises(ValueError, match="q_rope"):
        spa.sparse_attn_latent_decode(t(3, 2, 64), None, p, pos, scale=1.0)
    with pytest.raises(ValueError, match="out"):
        spa.sparse_attn_latent_decode(t(3, 2, 64), t(3, 2, 16), p, pos, scale=1.0, out=t(3, 2, 80))
    with pytest.raises(ValueError, match="num_seqs"):
        spa.sparse_attn_latent_decode(t(3, 2, 64), t(3, 2, 16), p, pos, scale=1.0, num_seqs=2)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="agree"):
        spa.sparse_attn_latent_prefill(t(3, 2, 24), t(3, 1, 16), t(3, 8), t(3, 2, 16), cu, cu, scale=1.0)
    with pytest.raises(ValueError, match="k_rope"):
        spa.sparse_attn_latent_prefill(t(3, 2, 24), t(3, 2, 16), None, t(3, 2, 16), cu, cu, scale=1.0)
    with pytest.raises(ValueError, match="cu_k"):
        spa.sparse_attn_latent_prefill(t(3, 2, 24), t(3, 2, 16), t(3, 8), t(3, 2, 16), cu, cu[:1], scale=1.0)
    with pytest.raises(ValueError, match="CUDA"):
        spa.sparse_attn_latent_prefill(t(3, 2, 24), t(3, 2, 16), t(3, 8), t(3, 2, 16), cu, cu, scale=1.0)
