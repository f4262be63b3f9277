"""The order of the latent kernels' waits, on the CPU: every interleaving of a CTA's warps is walked
with the rings that the kernels use (tests/latent_order.cpp, csrc/spa_latent_ring.h).  A wait by parity
must never stand more than one phase from its barrier: earlier it would pass at once, later it would
hold for a phase that has gone by.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("order") / "latent_order")
    r = subprocess.run([cxx, "-std=c++17", "-O2", "-I",
                        os.path.join(ROOT, "sparse_paged_attention_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "latent_order.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(*args):
        return subprocess.run([exe, *[str(a) for a in args]], capture_output=True, text=True,
                              check=True, timeout=300).stdout.strip()
    return run


# tiles of each token; bit k of a mask: the running maximum moves at tile k (O is rescaled then)
TOKENS = [[1], [3], [7], [1, 1, 1, 1], [3, 3], [4, 2], [1, 5], [2, 1, 3]]
MASKS = [0, 0x7F, 0x2A, 0x15]


@pytest.mark.parametrize("boxed", [0, 1])
@pytest.mark.parametrize("fp8", [0, 1])
@pytest.mark.parametrize("tiles", TOKENS, ids=str)
def test_decode_waits_are_within_a_phase(order, tiles, fp8, boxed):
    for mask in MASKS:
        assert order("decode", fp8, boxed, 0, mask, *tiles).startswith("ok"), (mask, tiles)


def test_two_barriers_over_three_buffers_are_not_enough(order):
    """What the walk is for: with P-ready and PV-done barriers in rings of two, as they once were, the
    bf16 softmax reads O before the products of the last tiles, where no maximum moved; the e4m3 one,
    which waits for the tile before the last, does not."""
    for tiles in ([3], [3, 2], [7]):
        assert order("decode", 0, 1, 2, 0, *tiles).startswith("early at softmax, PV_DONE"), tiles
        assert order("decode", 1, 1, 2, 0, *tiles).startswith("ok"), tiles


# items of a CTA: key steps of the first and the second query tile, and whether the last ends in a tile
ITEMS = ["1,0,1", "2,0,1", "0,1,1", "1,1,1", "1,2,1", "2,2,0", "2,3,1"]


def item_lists(n):
    lists = [[]]
    for _ in range(n):
        lists = [x + [i] for x in lists for i in ITEMS]
    return [x for x in lists if sum(max(map(int, i.split(",")[:2])) for i in x) <= 4]


@pytest.mark.parametrize("first", ITEMS)
def test_prefill_waits_are_within_a_phase(order, first):
    for items in [x for n in (1, 2) for x in item_lists(n) if x[0] == first]:
        assert order("prefill", 1, 1, *items).startswith("ok"), items


def test_prefill_waits_with_three_chunks_a_key(order):
    for items in (["2,3,1"], ["2,0,1", "0,1,1"]):
        assert order("prefill", 3, 1, *items).startswith("ok"), items


def test_prefill_without_the_loaders_wait_is_early(order):
    """An item of one query tile, then one whose first query tile sees no key: without the loader's
    wait, the second query tile's wait for V may be two phases from its barrier."""
    for items in (["2,0,1", "0,1,1"], ["1,0,1", "2,0,1", "0,1,1"]):
        for chunks in (1, 3):
            assert order("prefill", chunks, 0, *items).startswith("early at softmax 1, V_FULL"), items
            assert order("prefill", chunks, 1, *items).startswith("ok"), items
