"""Rotation, norms, appends and tree decode: what the entry points refuse on the host, before touching a GPU
(CPU only)."""
import ctypes
import os

import pytest
import torch

import sparse_paged_attention_gb300 as spa
from sparse_paged_attention_gb300 import (SpaAppendC, SpaHeadRowsC, SpaLatentPoolC, SpaLatentTreeC, SpaPoolC,
                                          SpaRopeProblemC)

S = spa.SPA_STATUS


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses: host validation is tested without a GPU")
    if not os.path.exists(spa.library_path()):
        from sparse_paged_attention_gb300.build import build_library
        build_library()
    return spa.load_library()


def rows(**kw):
    f = dict(x=0x10000, out=0x20000, weight=None, x_stride_t=512, x_stride_h=64, out_stride_t=512, out_stride_h=64,
             num_heads=8, reserved=0)
    f.update(kw)
    return SpaHeadRowsC(*[f[n] for n, _ in SpaHeadRowsC._fields_])


def rope(lib, norm=False, q=None, k=None, **kw):
    f = dict(num_tokens=4, head_dim=64, rope_dim=32, rope_start=32, interleaved=1, inverse=0, weight_dtype=0,
             reserved=0, rope_scale=1.0, eps=1e-6, positions=0x30000, turns=0x40000)
    f.update(kw)
    p = SpaRopeProblemC(*[f[n] for n, _ in SpaRopeProblemC._fields_[:-2]])
    p.q, p.k = rows(**(q or {})), rows(**(k or dict(num_heads=0)))
    return (lib.sparse_attn_norm_rope if norm else lib.sparse_attn_rope)(ctypes.byref(p), None)


def test_structs_are_packed_as_declared():
    for name, c in (("_ROPE", SpaRopeProblemC), ("_APPEND", SpaAppendC), ("_LATENT_TREE", SpaLatentTreeC)):
        assert getattr(spa, name).size == ctypes.sizeof(c)


@pytest.mark.parametrize("norm", [False, True])
def test_rope_refusals(lib, norm):
    def says(code, **kw):
        assert rope(lib, norm, **kw) == S[code], kw
    assert (lib.sparse_attn_norm_rope if norm else lib.sparse_attn_rope)(None, None) == S["SPA_ERR_NULL"]
    for bad in (dict(num_tokens=-1), dict(head_dim=0), dict(rope_dim=-8), dict(rope_start=-8), dict(rope_start=40),
                dict(rope_scale=float("nan")), dict(q=dict(num_heads=-1)), dict(q=dict(x_stride_t=-8)),
                dict(q=dict(out_stride_h=56)), dict(q=dict(out_stride_t=0)),
                dict(q=dict(out=0x10000, out_stride_h=72, out_stride_t=576))):
        says("SPA_ERR_SHAPE", **bad)
    for bad in (dict(head_dim=68), dict(head_dim=1032), dict(rope_dim=12), dict(rope_start=12),
                dict(num_tokens=1 << 28)):
        says("SPA_ERR_UNSUPPORTED", **bad)
    for bad in (dict(positions=None), dict(turns=None), dict(q=dict(x=None)), dict(k=dict(out=None))):
        says("SPA_ERR_NULL", **bad)
    for bad in (dict(q=dict(x=0x10008)), dict(k=dict(out=0x20004)), dict(q=dict(x_stride_h=68)), dict(turns=0x40004)):
        says("SPA_ERR_ALIGN", **bad)
    says("SPA_OK", num_tokens=0)
    says("SPA_OK", q=dict(num_heads=0))
    # the call then stops at the device query
    says("SPA_ERR_CUDA")
    says("SPA_ERR_CUDA", rope_dim=0, turns=None, q=dict(out=0x10000))
    if norm:
        for bad in (dict(eps=0.0), dict(eps=float("inf")), dict(weight_dtype=2)):
            says("SPA_ERR_SHAPE", **bad)
        says("SPA_ERR_ALIGN", q=dict(weight=0x50004))


def append(lib, pool, fp8=False, **kw):
    latent = isinstance(pool, SpaLatentPoolC)
    f = dict(num_tokens=5, num_seqs=2, head_dim=512, rope_dim=64, rope_start=0, interleaved=1, norm=1, weight_dtype=1,
             rope_scale=1.0, eps=1e-6, positions=0x60000, entries=None, seq_of_token=None, turns=0x70000, k=0x80000,
             v=0x90000, weight=0xA0000, k_stride=576, v_stride=576)
    f.update(kw)
    p = SpaAppendC(*[f[n] for n, _ in SpaAppendC._fields_])
    name = "sparse_attn_%s_append%s" % ("latent" if latent else "paged_kv", "_fp8" if fp8 else "")
    return getattr(lib, name)(ctypes.byref(p), ctypes.byref(pool), None)


def kv_pool(**kw):
    f = dict(kv=0x10000, k_scale=0x20000, v_scale=0x30000, block_table=0x40000, num_blocks=64, page_size=64, bt_stride=8)
    f.update(kw)
    return SpaPoolC(*[f[n] for n, _ in SpaPoolC._fields_])


def latent_pool(**kw):
    f = dict(rows=0x10000, scale=0x20000, block_table=0x30000, num_blocks=64, page_size=64, bt_stride=8, latent_dim=512,
             rope_dim=64)
    f.update(kw)
    return SpaLatentPoolC(*[f[n] for n, _ in SpaLatentPoolC._fields_])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("pool", [kv_pool, latent_pool])
def test_append_refusals(lib, pool, fp8):
    def says(code, p=None, **kw):
        assert append(lib, pool() if p is None else p, fp8, **kw) == S[code], kw
    for bad in (dict(num_tokens=-1), dict(num_seqs=0), dict(rope_dim=-8), dict(rope_scale=float("inf")),
                dict(k_stride=-8), dict(v_stride=-8), dict(eps=0.0), dict(eps=-1.0), dict(weight_dtype=3)):
        says("SPA_ERR_SHAPE", **bad)
    for bad in (dict(positions=None), dict(turns=None), dict(k=None), dict(v=None)):
        says("SPA_ERR_NULL", **bad)
    for bad in (dict(k=0x80008), dict(v=0x90008), dict(k_stride=516), dict(v_stride=68), dict(weight=0xA0004)):
        says("SPA_ERR_ALIGN", **bad)
    says("SPA_ERR_SHAPE", pool(num_blocks=0))
    says("SPA_ERR_UNSUPPORTED", pool(num_blocks=1 << 25))
    says("SPA_ERR_NULL", pool(block_table=None))
    says("SPA_OK", num_tokens=0)
    says("SPA_ERR_CUDA")
    says("SPA_ERR_CUDA", norm=0, eps=0.0, weight=None)
    if pool is kv_pool:
        says("SPA_ERR_UNSUPPORTED", head_dim=96)
        says("SPA_ERR_UNSUPPORTED", head_dim=576)
        says("SPA_ERR_SHAPE", rope_start=456)
        says("SPA_ERR_ALIGN", kv_pool(kv=0x10008))
        if fp8:
            says("SPA_ERR_NULL", kv_pool(v_scale=None))
    else:
        for bad in (dict(head_dim=448), dict(rope_dim=32), dict(rope_start=8)):
            says("SPA_ERR_SHAPE", **bad)
        says("SPA_ERR_UNSUPPORTED", latent_pool(latent_dim=96))


def tree(lib, pool, fp8=False, out=0xE0000, ws=0xF0000, wb=1 << 40, **kw):
    f = dict(num_tokens=6, num_seqs=2, num_heads=64, mask_words=1, scale=0.07, reserved=0, context_lens=0x60000,
             cu_tokens=0x70000, tree_mask=0x80000, q_latent=0x90000, q_rope=0xA0000, q_latent_stride_t=64 * 512,
             q_latent_stride_h=512, q_rope_stride_t=64 * 64, q_rope_stride_h=64)
    f.update(kw)
    p = SpaLatentTreeC(*[f[n] for n, _ in SpaLatentTreeC._fields_])
    fn = lib.sparse_attn_latent_tree_decode_fp8 if fp8 else lib.sparse_attn_latent_tree_decode
    return fn(ctypes.byref(pool), ctypes.byref(p), out, ws, wb, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_refusals(lib, fp8):
    def says(code, p=None, **kw):
        assert tree(lib, latent_pool() if p is None else p, fp8, **kw) == S[code], kw
    for bad in (dict(num_tokens=-1), dict(num_seqs=-1), dict(num_heads=0), dict(mask_words=0), dict(mask_words=-1),
                dict(scale=float("nan")), dict(q_latent_stride_t=-8), dict(q_latent_stride_h=504),
                dict(q_rope_stride_t=56)):
        says("SPA_ERR_SHAPE", **bad)
    says("SPA_ERR_UNSUPPORTED", num_tokens=1 << 20, num_heads=1 << 11)
    for bad in (dict(context_lens=None), dict(cu_tokens=None), dict(q_latent=None), dict(q_rope=None), dict(out=None)):
        says("SPA_ERR_NULL", **bad)
    for bad in (dict(q_latent=0x90008), dict(q_rope=0xA0002), dict(q_latent_stride_h=516), dict(out=0xE0008)):
        says("SPA_ERR_ALIGN", **bad)
    says("SPA_ERR_UNSUPPORTED", latent_pool(rope_dim=72))
    says("SPA_ERR_SHAPE", latent_pool(page_size=0))
    says("SPA_OK", num_tokens=0)
    says("SPA_OK", num_seqs=0)
    says("SPA_ERR_CUDA")
    says("SPA_ERR_CUDA", tree_mask=None, mask_words=0)
    assert lib.sparse_attn_latent_tree_decode_workspace_size(None, ctypes.byref(latent_pool())) == 0


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("which", ["q", "k"])
def test_output_rows_that_overlap_are_refused(lib, norm, which):
    """Each stride alone leaves room for a row, but rows of several tokens and heads fall on one another."""
    def says(code, T=4, **kw):
        assert rope(lib, norm, num_tokens=T, **{which: kw}) == S[code], kw
    for bad in (dict(out_stride_t=64), dict(out_stride_t=504), dict(out_stride_t=64, out_stride_h=248),
                dict(out_stride_t=1 << 37, out_stride_h=1 << 36)):
        says("SPA_ERR_SHAPE", **bad)
    # tokens behind all heads, heads behind all tokens, and one token or head
    for good in (dict(), dict(out_stride_t=64, out_stride_h=256), dict(out_stride_t=1 << 37, out_stride_h=1 << 34),
                 dict(out_stride_t=64, num_heads=1)):
        says("SPA_ERR_CUDA", **good)
    says("SPA_ERR_CUDA", T=1, out_stride_t=64)
    says("SPA_ERR_SHAPE", T=1 << 20, out_stride_t=1 << 37, out_stride_h=1 << 38)   # (their product passes 64 bits)
