"""Latent attention: what the Python layer refuses before the library is called, on tensors that only
claim a device (CPU only: nothing is launched)."""
import pytest
import torch

import sparse_paged_attention_gb300 as spa


class OnDevice(torch.Tensor):
    """A host tensor that says it is on GPU `index`."""
    index = 0

    def get_device(self):
        return self.index


class OnOtherDevice(OnDevice):
    index = 1


def claim(t, cls=OnDevice):
    return t.as_subclass(cls)


def zeros(*shape, dtype=torch.bfloat16):
    return claim(torch.zeros(shape, dtype=dtype))


def pools(block_table):
    return (spa.LatentPool(zeros(4, 8, 80), block_table, 16),
            spa.LatentPool(zeros(4, 8, 96, dtype=torch.uint8), block_table, 16,
                           zeros(32, dtype=torch.float32)))


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    """The library is not there to be called."""
    monkeypatch.setattr(spa, "load_library", lambda: None)


@pytest.mark.parametrize("where", ["host", "another GPU"])
def test_block_table_elsewhere_is_refused(where):
    bt = torch.zeros((1, 4), dtype=torch.int32)
    if where != "host":
        bt = claim(bt, OnOtherDevice)
    pos = zeros(3, dtype=torch.int32)
    bf16, e4m3 = pools(bt)
    for pool, write, read, decode in (
            (bf16, spa.sparse_attn_latent_write, spa.sparse_attn_latent_read, spa.sparse_attn_latent_decode),
            (e4m3, spa.sparse_attn_latent_write_fp8, spa.sparse_attn_latent_read_fp8,
             spa.sparse_attn_latent_decode_fp8)):
        with pytest.raises(ValueError, match="block_table"):
            write(zeros(3, 64), zeros(3, 16), pos, pool)
        with pytest.raises(ValueError, match="block_table"):
            read(pos, pool)
        with pytest.raises(ValueError, match="block_table"):
            decode(zeros(3, 2, 64), zeros(3, 2, 16), pool, pos, scale=1.0)
        with pytest.raises(ValueError, match="block_table"):
            spa.bind_latent_decode(zeros(3, 2, 64), zeros(3, 2, 16), pool, pos, scale=1.0,
                                   fp8=pool is e4m3)
        with pytest.raises(ValueError, match="block_table"):
            spa.sparse_attn_latent_decode_workspace_size(zeros(3, 2, 64), pool, pos, fp8=pool is e4m3)
