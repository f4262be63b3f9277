"""Rotation, norms, appends and tree decode: what the Python layer refuses before the library is called, and which
stream's memory a call takes, on tensors that only claim a device (CPU only: nothing is launched)."""
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from test_latent_binding import OnOtherDevice, claim, device, pools, zeros  # noqa: F401

i32 = dict(dtype=torch.int32)


def table(n=8, cls=None):
    t = torch.zeros(n, dtype=torch.int64)
    return spa.RotaryTable(claim(t) if cls is None else claim(t, cls))


@pytest.mark.parametrize("given", [None, 7, 9, "object", 0])
def test_memory_comes_from_the_stream_of_the_call(device, given, monkeypatch):  # noqa: F811
    lib, made, Stream = device
    new = torch.Tensor.new_empty

    def note_new(self, shape, **kw):
        made.append(torch.cuda.current_stream().cuda_stream)
        return claim(new(self, shape, **kw))
    monkeypatch.setattr(torch.Tensor, "new_empty", note_new)
    stream = Stream(9) if given == "object" else given
    want = 7 if given is None else 9 if given == "object" else given
    pos, cu, bt = zeros(3, **i32), zeros(2, **i32), zeros(1, 4, **i32)
    spa.sparse_attn_rope(zeros(3, 2, 64), pos, table(), stream=stream)
    spa.sparse_attn_norm_rope(zeros(3, 2, 64), zeros(3, 1, 64), pos, table(), stream=stream)
    assert len(made) >= 3 and set(made) == {want} and lib.streams == [want] * 2
    kv = (spa.PagedPool(zeros(4, 8, 2, 64), bt),
          spa.PagedPool(zeros(4, 8, 2, 64, dtype=torch.uint8), bt, zeros(32, dtype=torch.float32),
                        zeros(32, dtype=torch.float32)))
    for pool, lat, suffix in zip(kv, pools(bt), ("", "_fp8")):
        made.clear()
        lib.streams.clear()
        getattr(spa, "sparse_attn_paged_kv_append" + suffix)(zeros(3, 64), zeros(3, 64), pos, pool, table(), stream=stream)
        getattr(spa, "sparse_attn_latent_append" + suffix)(zeros(3, 64), zeros(3, 16), pos, lat, table(), stream=stream)
        args = (zeros(3, 2, 64), zeros(3, 2, 16), lat, zeros(1, **i32), cu, zeros(3, 1, **i32))
        getattr(spa, "sparse_attn_latent_tree_decode" + suffix)(*args, scale=1.0, stream=stream)
        spa.bind_latent_tree_decode(*args, scale=1.0, fp8=bool(suffix), stream=stream)()
        assert made == [want] * 4 and lib.streams == [want] * 4      # out and workspace of both


def test_refusals(device):  # noqa: F811
    other = lambda *s, **kw: claim(torch.zeros(s, **(kw or dict(dtype=torch.bfloat16))), OnOtherDevice)  # noqa: E731
    x, pos, bt = zeros(3, 2, 64), zeros(3, **i32), zeros(1, 4, **i32)
    for call in (
            lambda: spa.sparse_attn_rope(x, other(3, **i32), table()),
            lambda: spa.sparse_attn_rope(x, pos, table(cls=OnOtherDevice)),
            lambda: spa.sparse_attn_rope(x, pos, table(), out=other(3, 2, 64)),
            lambda: spa.sparse_attn_rope(other(3, 2, 64), other(3, **i32), table(cls=OnOtherDevice)),   # not the current one
            lambda: spa.sparse_attn_rope(torch.zeros((3, 2, 64), dtype=torch.bfloat16), pos, table()),
            lambda: spa.sparse_attn_rope(x[..., ::2], pos, table()),
            lambda: spa.sparse_attn_norm_rope(x, zeros(3, 1, 32), pos, table()),
            lambda: spa.sparse_attn_norm_rope(x, None, pos, table(), q_weight=zeros(64, dtype=torch.float16)),
            lambda: spa.sparse_attn_norm_rope(x, x, pos, table(), q_weight=zeros(64),
                                              k_weight=zeros(64, dtype=torch.float32))):
        with pytest.raises(ValueError):
            call()
    kv = spa.PagedPool(zeros(4, 8, 2, 64), bt)
    for bad in (dict(k=zeros(2, 64)), dict(v=zeros(3, 32)), dict(entries=zeros(2, **i32)), dict(entries=zeros(3)),
                dict(weight=zeros(64)), dict(weight=zeros(32), eps=1e-6), dict(num_seqs=2), dict(positions=zeros(2, **i32)),
                dict(entries=other(3, **i32)), dict(seq_of_token=zeros(2, **i32))):
        kw = dict(k=zeros(3, 64), v=zeros(3, 64), positions=pos, pool=kv, table=table(), **{})
        kw.update(bad)
        with pytest.raises(ValueError):
            spa.sparse_attn_paged_kv_append(**kw)
    for lat, suffix in zip(pools(bt), ("", "_fp8")):
        for latent, rope, tab in ((zeros(3, 32), zeros(3, 16), table()), (zeros(3, 64), None, table()),
                                  (zeros(3, 64), zeros(3, 16), None), (zeros(3, 64), zeros(3, 16), table(4)),
                                  (zeros(3, 64), zeros(2, 16), table())):
            with pytest.raises(ValueError):
                getattr(spa, "sparse_attn_latent_append" + suffix)(latent, rope, pos, lat, tab)
    e4m3 = spa.PagedPool(zeros(4, 8, 2, 64, dtype=torch.uint8), bt, zeros(32, dtype=torch.float32),
                         zeros(31, dtype=torch.float32))
    with pytest.raises(ValueError):
        spa.sparse_attn_paged_kv_append_fp8(zeros(3, 64), zeros(3, 64), pos, e4m3, table())
    assert device[0].streams == []
