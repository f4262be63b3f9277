"""The Python layer of latent attention on the GPU: block tables on the host."""
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from test_gpu_latent import dev, place  # noqa: F401
from workloads import latent_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_block_table_on_the_host_is_refused(dev, fp8):  # noqa: F811
    inp = latent_inputs([20], 64, 16, 16, seed=64)
    pool, *_ = place(inp, fp8, dev)
    pool = pool._replace(block_table=pool.block_table.cpu())
    pos = torch.zeros(1, dtype=torch.int32, device=dev)
    x = torch.zeros((1, 4, 80), dtype=torch.bfloat16, device=dev)
    suffix = "_fp8" if fp8 else ""
    for call in (lambda: getattr(spa, "sparse_attn_latent_write" + suffix)(x[:, 0, :64], x[:, 0, 64:], pos, pool),
                 lambda: getattr(spa, "sparse_attn_latent_read" + suffix)(pos, pool),
                 lambda: getattr(spa, "sparse_attn_latent_decode" + suffix)(x[..., :64], x[..., 64:], pool, pos,
                                                                            scale=1.0)):
        with pytest.raises(ValueError, match="block_table"):
            call()
