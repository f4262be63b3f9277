"""The order of the tree decode kernel's waits, on the CPU: every interleaving of its warps is walked
(tests/latent_tree_order.cpp).  A wait by parity never stands more than one phase from its barrier, and no
state is one in which all are stuck."""
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
    exe = str(tmp_path_factory.mktemp("order") / "latent_tree_order")
    r = subprocess.run([cxx, "-std=c++17", "-O2", "-I", os.path.join(ROOT, "sparse_paged_attention_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "latent_tree_order.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(tiles, box=1, qtma=1, early=1, grow=0, k=(1, 1), v=(1, 1), soft=1):
        args = [box, qtma, early, grow, *k, *v, soft, *tiles]
        return subprocess.run([exe, *[str(a) for a in args]], capture_output=True, text=True, check=True,
                              timeout=300).stdout.strip()
    return run


@pytest.mark.parametrize("case", [
    dict(tiles=[2], k=(3, 3), v=(4, 3), soft=2), dict(tiles=[1, 1], v=(4, 3), soft=2), dict(tiles=[2, 1], v=(4, 3)),
    dict(tiles=[3], grow=6, v=(2, 2), soft=2), dict(tiles=[6], grow=42), dict(tiles=[2, 3, 1], v=(2, 1)),
    dict(tiles=[2, 1], k=(2, 2)), dict(tiles=[1, 1, 1], qtma=0, v=(2, 2)),
    dict(tiles=[6], box=0), dict(tiles=[1, 3], box=0, qtma=0, v=(2, 1)), dict(tiles=[2, 1], box=0, k=(3, 3), v=(4, 2))],
    ids=str)
def test_waits_are_within_a_phase(order, case):
    assert order(**case).startswith("ok")


def test_maxima_always_a_tile_ahead_would_be_stuck(order):
    """What the walk is for: the first tile of a unit waits for q, which comes after the last tile's V, which may
    wait for that tile's P; so its maxima must not come before that P."""
    assert order([1, 1], early=2, v=(4, 3), soft=2).startswith("stuck")
    assert order([2], early=2, box=0, v=(4, 2)).startswith("stuck")
