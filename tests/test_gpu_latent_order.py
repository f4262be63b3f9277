"""The latent kernels where their warps run ahead of one another as far as the rings allow: decode in
parts of a few tiles, calls back to back; prefill items with and without a second query tile in turn."""
import pytest
import torch

import sparse_paged_attention_gb300 as spa
from test_gpu_latent import decode_case, dev, prefill_case  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tiles", [3, 4, 7])
def test_decode_parts_of_a_few_tiles_repeat(dev, tiles, fp8):  # noqa: F811
    """One sequence cut into parts of `tiles` 64-entry tiles, one a slice of the device's SMs (128 heads:
    two groups a slice).  The scores are alike, so that after a part's first tile no maximum moves far
    enough for a rescale, which would wait for the product of the tile before."""
    slices = torch.cuda.get_device_properties(dev).multi_processor_count // 2
    n, H, L, R = 64 * tiles * slices - 5, 128, 128, 16
    pool, ql, qr, pos, sid, out = decode_case(dev, [n], H, L, R, 64, fp8, seed=70 + tiles, scale=0.01)
    call = spa.bind_latent_decode(ql.to(dev), qr.to(dev), pool, pos.to(dev), fp8=fp8, scale=0.01,
                                  seq_of_token=sid.to(dev))
    outs = []
    for _ in range(50):
        call()
        outs.append(call.out.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            call()
    for _ in range(10):
        call.out.zero_()
        graph.replay()
        outs.append(call.out.clone())
    for x in outs:
        assert torch.equal(x.view(torch.int16), out.view(torch.int16))


def test_prefill_items_of_one_query_tile_and_of_none(dev):  # noqa: F811
    """As many heads as SMs, so that a CTA's items are the sequences in turn: one query tile of several
    key steps, then one whose first query tile sees no key and whose second ends inside a tile."""
    H = torch.cuda.get_device_properties(dev).multi_processor_count
    nq, nk = [100, 200, 90, 170, 128, 250], [300, 50, 400, 40, 257, 120]
    rows = {0, 99, 100, 249, 250, 299, 300, 389, 390, 519, 520, 559, 560, 687, 688, 818, 937}
    first = prefill_case(dev, nq, nk, H, 32, 16, 32, seed=81, rows=rows)
    for _ in range(10):
        again = prefill_case(dev, nq, nk, H, 32, 16, 32, seed=81, rows=set())
        assert (again == first).all()
