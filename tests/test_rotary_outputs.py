"""Outputs of norm + rotation that would be written while the other tensor is read or written (CPU only: nothing is
launched)."""
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from test_latent_binding import claim, device, zeros  # noqa: F401


def test_outputs_on_the_other_tensor_are_refused(device):  # noqa: F811
    pos, table = zeros(3, dtype=torch.int32), spa.RotaryTable(claim(torch.zeros(8, dtype=torch.int64)))
    q, k, o = (zeros(3, 2, 64) for _ in range(3))
    fused = zeros(3, 5, 64)
    for kw in (dict(q_out=o, k_out=o), dict(q_out=k), dict(k_out=q), dict(q_out=k, k_out=q), dict(q_out=q, k_out=q),
               dict(q=fused[:, :3], k=fused[:, 3:], q_out=fused[:, 1:4], k_out=o),
               dict(q=fused[:, :3], k=fused[:, 3:], q_out=fused[:, :3], k_out=fused[:, 2:4]),
               dict(q=q, k=q, q_out=q), dict(q_out=fused[:, :2], k_out=fused[:, 1:3])):
        args = dict(dict(q=q, k=k, positions=pos, table=table), **kw)
        with pytest.raises(ValueError, match="overlap"):
            spa.sparse_attn_norm_rope(**args)
    lib = device[0]
    assert lib.streams == []
    for kw in (dict(), dict(q_out=q, k_out=k), dict(q_out=o), dict(k_out=o), dict(q=q, k=q), dict(q_out=q),
               dict(q=fused[:, :3], k=fused[:, 3:], q_out=fused[:, :3], k_out=fused[:, 3:]),
               dict(q_out=fused[:, :2], k_out=fused[:, 2:4]), dict(q_out=fused[:, 3:], k_out=fused[:, :2]),
               dict(k=None, q_out=q),
               dict(q=zeros(0, 2, 64), k=zeros(0, 2, 64), positions=zeros(0, dtype=torch.int32), q_out=zeros(0, 2, 64),
                    k_out=zeros(0, 2, 64))):
        spa.sparse_attn_norm_rope(**dict(dict(q=q, k=k, positions=pos, table=table), **kw))
    # heads of q and k in turn within one buffer
    turns = zeros(3, 4, 64)
    spa.sparse_attn_norm_rope(turns[:, ::2], turns[:, 1::2], pos, table, q_out=turns[:, ::2], k_out=turns[:, 1::2])
    # and with heads before tokens
    heads = zeros(4, 3, 64).transpose(0, 1)
    spa.sparse_attn_norm_rope(heads[:, :2], heads[:, 2:], pos, table, q_out=heads[:, :2], k_out=heads[:, 2:])
    with pytest.raises(ValueError, match="overlap"):
        spa.sparse_attn_norm_rope(heads[:, :2], heads[:, 2:], pos, table, q_out=heads[:, 1:3], k_out=o)
    assert len(lib.streams) == 13
