"""Which stream the memory of a call comes from, for the entry points of paged attention (CPU only: the
library and the device are stand-ins)."""
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from test_latent_binding import claim, device, zeros  # noqa: F401

i32 = dict(dtype=torch.int32)


@pytest.mark.parametrize("given", [None, 7, 9, "object", 0])
def test_memory_comes_from_the_stream_of_the_call(device, given, monkeypatch):  # noqa: F811
    lib, made, Stream = device

    def note(name):
        make = getattr(torch, name)

        def made_here(*args, device=None, **kw):
            made.append(torch.cuda.current_stream().cuda_stream)
            return claim(make(*args, **kw))
        monkeypatch.setattr(torch, name, made_here)
    note("full")
    note("empty_like")
    stream = Stream(9) if given == "object" else given
    want = 7 if given is None else 9 if given == "object" else given
    pool = spa.PagedPool(zeros(4, 8, 2, 64), zeros(1, 4, **i32))
    q, pos, topk = zeros(3, 2, 64), zeros(3, **i32), zeros(3, 8, **i32)
    kw = dict(window=16, ratio=4, stream=stream)
    args = (q, pool, pool, topk, pos)
    logits = zeros(3, 40, dtype=torch.float32)
    calls = [
        (lambda: spa.sparse_attn_paged_prefill(*args, scale=1.0, **kw), 1),
        (lambda: spa.bind_prefill(*args, scale=1.0, **kw)(), 1),
        (lambda: spa.sparse_attn_paged_decode(*args, scale=1.0, **kw), 2),
        (lambda: spa.bind_decode(*args, scale=1.0, **kw)(), 2),
        (lambda: spa.sparse_attn_paged_decode_noalloc(*args, scale=1.0, **kw), 1),
        (lambda: spa.sparse_attn_paged_resolve_columns(pool, pool, topk, pos, **kw), 1),
        (lambda: spa.sparse_attn_gated_pool(zeros(2, 4, 8, dtype=torch.float32),
                                            zeros(2, 4, 8, dtype=torch.float32), stream=stream), 1),
        (lambda: spa.sparse_attn_indexer_logits(zeros(3, 2, 128), zeros(3, 2, dtype=torch.float32),
                                                zeros(4, 8, 17, **i32), zeros(1, 4, **i32), pos, ratio=4,
                                                num_cols=8, stream=stream), 1),
        (lambda: spa.sparse_attn_indexer_topk(logits, 4, stream=stream), 1),
    ]
    for call, tensors in calls:
        made.clear()
        call()
        # (resolve_columns also has a stand-in for q, which is no device memory)
        assert len(made) >= tensors and made[:tensors] == [want] * tensors
    assert lib.streams == [want] * len(calls)
