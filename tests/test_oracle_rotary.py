"""The rotary and tree oracles against closed forms and brute force (CPU only), and the frequency tables."""
import math

import numpy as np
import pytest

import sparse_paged_attention_gb300 as spa
from oracle import latent as olat
from oracle import latent_tree as otree
from oracle import rotary as orot


def quarter():
    return [1 << 62]          # a quarter of a turn a position


@pytest.mark.parametrize("interleaved", [True, False])
def test_quarter_turns(interleaved):
    x = np.array([[3.0, 5.0, 7.0]])
    want = {0: (3, 5), 1: (-5, 3), 2: (-3, -5), 3: (5, -3), -1: (5, -3), 4 * 10 ** 8 + 1: (-5, 3)}
    for p, (a, b) in want.items():
        y = orot.rotate(x, [p], quarter(), start=0, interleaved=interleaved)
        assert np.allclose(y, [[a, b, 7.0]], atol=1e-12), p


def test_layouts_inverse_and_relative_positions():
    rng = np.random.default_rng(0)
    turns = [int(t) for t in rng.integers(-(1 << 62), 1 << 62, 4)]
    x, y = rng.standard_normal((2, 1, 12))
    for il in (True, False):
        kw = dict(start=4, interleaved=il)
        back = orot.rotate(orot.rotate(x, [77], turns, scale=2.0, **kw), [77], turns, inverse=True, scale=0.5, **kw)
        assert np.allclose(back, x)
        # products depend on the distance alone
        dot = [np.sum(orot.rotate(x, [p + 9], turns, **kw) * orot.rotate(y, [p], turns, **kw)) for p in (0, 3, 10 ** 6)]
        assert np.allclose(dot, dot[0])
    perm = [0, 1, 2, 3] + [4 + 2 * i for i in range(4)] + [5 + 2 * i for i in range(4)]
    a = orot.rotate(x, [5], turns, start=4, interleaved=True)[:, perm]
    assert np.allclose(a, orot.rotate(x[:, perm], [5], turns, start=4, interleaved=False))


def test_norm():
    y = orot.norm(np.array([[3.0, 4.0]]), [2.0, 1.0], 0.0)
    assert np.allclose(y, [[6.0 / math.sqrt(12.5), 4.0 / math.sqrt(12.5)]])


def radians(table):
    return np.array([t % (1 << 64) for t in table.turns.tolist()], dtype=np.float64) / 2.0 ** 64 * 2.0 * math.pi


def test_tables():
    part = dict(rtol=1e-14, atol=2 * math.pi * 2.0 ** -65)    # half of a turn's 2^64 parts
    plain = spa.sparse_attn_rotary_table(64, device="cpu")
    f = 10000.0 ** (-np.arange(32) / 32.0)
    assert plain.scale == 1.0 and np.allclose(radians(plain), f, **part)
    lin = spa.sparse_attn_rotary_table(64, scaling="linear", factor=4.0, device="cpu")
    assert np.allclose(radians(lin), f / 4, **part)
    ntk = spa.sparse_attn_rotary_table(64, scaling="ntk", factor=4.0, device="cpu")
    assert np.allclose(radians(ntk)[[0, 31]], [1.0, f[31] / 4], rtol=1e-12, atol=0)
    yarn = spa.sparse_attn_rotary_table(64, scaling="yarn", factor=16.0, original_length=4096, device="cpu")
    g = radians(yarn)
    turns = 4096 * f / (2 * math.pi)
    assert np.allclose(g[turns > 36], f[turns > 36], **part)
    assert np.allclose(g[turns < 0.7], f[turns < 0.7] / 16, **part)
    assert np.all(np.diff(g) < 0) and np.all(g <= f * (1 + 1e-12)) and np.all(g >= f / 16 * (1 - 1e-12))
    assert yarn.scale == 0.1 * math.log(16.0) + 1.0
    own = spa.sparse_attn_rotary_table(4, inv_freq=[7.0, -0.25], scale=0.5, interleaved=False, device="cpu")
    assert np.allclose(radians(own), [7.0 - 2 * math.pi, 2 * math.pi - 0.25]) and own.scale == 0.5
    assert not own.interleaved
    for bad in (dict(rope_dim=7), dict(rope_dim=8, scaling="other"), dict(rope_dim=8, factor=0.0),
                dict(rope_dim=8, inv_freq=[1.0]), dict(rope_dim=2, scaling="ntk"),
                dict(rope_dim=8, scaling="yarn", beta_slow=0.0)):
        with pytest.raises(ValueError):
            spa.sparse_attn_rotary_table(device="cpu", **bad)


def test_trees_see_what_their_masks_name():
    assert otree.visible(2, 5, 3, [0b01010]) == [0, 1, 3, 5]
    assert otree.visible(1, 40, 3, [1 << 31, 0xFF]) == [0, 32, 33, 34, 35, 36, 37, 38, 39, 40]
    assert otree.visible(3, 5, 1, None) == [0, 1, 2, 3, 4]
    assert otree.visible(0, 3, 0, [0]) == []


def test_a_chain_is_the_decode_of_its_tokens():
    rng = np.random.default_rng(1)
    rows = rng.integers(0, 1 << 14, (4, 8, 12)).astype(np.uint16)      # small positive bf16 patterns
    bt = np.array([[2, 0], [3, 1]])
    q = rng.standard_normal((5, 2, 12))
    kw = dict(page_size=8, scale=0.3, fp8=False)
    got = otree.tree_decode(q[..., :8], q[..., 8:], [4, 0], [0, 2, 5], None, bt, rows, **kw)
    want, _ = olat.decode(q[..., :8], q[..., 8:], [4, 5, 0, 1, 2], [0, 0, 1, 1, 1], bt, rows, **kw)
    for t in range(5):
        assert np.allclose(got[t][0], want[t][0], rtol=1e-13)
