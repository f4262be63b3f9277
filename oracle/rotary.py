"""Rotary positions, norms of heads and the appends that do both.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain numpy, float64, from the definitions;
shares no code with the CUDA library.

* angle of pair i at position p: ``2 pi ((p * turns[i]) mod 2^64) / 2^64``, the product in integers;
* ``(a, b) -> m (a cos t - b sin t, b cos t + a sin t)``, pairs (2i, 2i + 1) or (i, i + R / 2);
* ``y = x / sqrt(mean(x^2) + eps) * w`` over the row.
"""
import math

import numpy as np


def angles(positions, turns) -> np.ndarray:
    """[T, R / 2] radians in [0, 2 pi)."""
    return np.array([[2.0 * math.pi * (((int(p) * int(t)) % (1 << 64)) / 2.0 ** 64) for t in turns]
                     for p in positions], dtype=np.float64).reshape(len(positions), len(turns))


def rotate(x, positions, turns, *, start: int, interleaved: bool, scale: float = 1.0,
           inverse: bool = False) -> np.ndarray:
    """x [T, .., D] float64, values start .. start + 2 len(turns) of every row rotated."""
    x = np.array(x, dtype=np.float64)
    R = 2 * len(turns)
    t = angles(positions, turns)
    t = t.reshape(t.shape[:1] + (1,) * (x.ndim - 2) + t.shape[1:])
    c, s = np.cos(t) * scale, np.sin(t) * (-scale if inverse else scale)
    at = start + np.arange(R // 2) * (2 if interleaved else 1)
    to = at + (1 if interleaved else R // 2)
    a, b = x[..., at].copy(), x[..., to].copy()
    x[..., at], x[..., to] = a * c - b * s, b * c + a * s
    return x


def norm(x, weight, eps: float) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return y if weight is None else y * np.asarray(weight, dtype=np.float64)


def pair_sizes(x, *, start: int, R: int, interleaved: bool) -> np.ndarray:
    """|a| + |b| of every rotated value's pair (0 elsewhere): the size of a rotation's terms."""
    out = np.zeros_like(np.asarray(x, dtype=np.float64))
    at = start + np.arange(R // 2) * (2 if interleaved else 1)
    to = at + (1 if interleaved else R // 2)
    z = np.abs(x[..., at]) + np.abs(x[..., to])
    out[..., at] = out[..., to] = z
    return out
