"""The Python layer of latent attention on the GPU: block tables on the host, calls on other streams."""
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from test_gpu_latent import decode_case, dev, place  # noqa: F401
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


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_calls_on_another_stream_keep_their_memory(dev, fp8, raw):  # noqa: F811
    """Calls on a side stream that is busy, and meanwhile allocations of the workspace's and the outputs'
    sizes on the current stream: neither side finds the other's bytes in its memory."""
    pool, ql, qr, pos, sid, want = decode_case(dev, [3000, 50], 64, 512, 64, 64, fp8, seed=45)
    suffix = "_fp8" if fp8 else ""
    decode = getattr(spa, "sparse_attn_latent_decode" + suffix)
    read = getattr(spa, "sparse_attn_latent_read" + suffix)
    args = (ql.to(dev), qr.to(dev), pool, pos.to(dev))
    kw = dict(scale=576 ** -0.5, seq_of_token=sid.to(dev))
    at = torch.arange(2000, dtype=torch.int32, device=dev)
    rows = read(at, pool)
    n = spa.sparse_attn_latent_decode_workspace_size(ql, pool, pos, fp8=fp8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    stream = side.cuda_stream if raw else side
    outs, held = [], []
    for _ in range(3):
        outs.append((decode(*args, stream=stream, **kw), read(at, pool, stream=stream)))
        for size in (n, want.numel() * 2, rows.numel() * 2):
            held.append(torch.full((size,), 0xA5, dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()
    for out, got in outs:
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        assert torch.equal(got.view(torch.int16), rows.view(torch.int16))
    assert all(bool((x == 0xA5).all()) for x in held)


@pytest.mark.parametrize("L,R,H", [(512, 64, 64), (64, 0, 16), (512, 8, 130), (448, 40, 20)])
def test_decode_workspace_is_what_the_header_says(dev, L, R, H):  # noqa: F811
    """bf16: no more for more tokens.  e4m3: the queries' codes on top, by the header's formula."""
    table = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    bf16 = spa.LatentPool(torch.zeros((1, 64, L + R), dtype=torch.bfloat16, device=dev), table, R)
    e4m3 = spa.LatentPool(torch.zeros((1, 64, L + 2 * R), dtype=torch.uint8, device=dev), table, R,
                          torch.ones(64, device=dev))

    def size(pool, tokens):
        return spa.sparse_attn_latent_decode_workspace_size(
            torch.empty((tokens, H, L), dtype=torch.bfloat16, device=dev), pool,
            torch.zeros(tokens, dtype=torch.int32, device=dev), fp8=pool is e4m3)
    codes = -(-H // 64) * (-(-(L + 2 * R) // 128) * 16384 + 256)
    parts = size(bf16, 1)
    for tokens in (1, 2, 7, 100):
        assert size(bf16, tokens) == parts
        assert parts + tokens * codes <= size(e4m3, tokens) < parts + tokens * codes + 256
