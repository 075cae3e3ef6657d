"""CPU oracle for rotary positions.

TEST INFRASTRUCTURE ONLY, under the same rule as ``oracle.attention``.

A pair (a, b) of a head at position p turns by the angle p f_i of its
frequency.  ``rotate`` is the definition in float64, as multiplication of
a + i b by factor e^(i p f).  ``rotate_f32`` takes the decisions the kernels
take: cosines and sines given as float32, two products and a sum per value,
each rounded to float32 -- for comparisons where the result is then rounded
to a few bits and has to agree bit for bit.
"""

from __future__ import annotations

import numpy as np

from .attention import as_float64, as_int64


def pair_dims(rot: int, offset: int, interleaved: bool):
    """(first, second) dims of pairs 0 .. rot / 2 - 1."""
    i = np.arange(rot // 2)
    if interleaved:
        return offset + 2 * i, offset + 2 * i + 1
    return offset + i, offset + i + rot // 2


def rotate(x, positions, inv_freq, *, factor: float = 1.0, interleaved: bool = False, offset: int = 0,
           inverse: bool = False) -> np.ndarray:
    """x [n, h, head_dim] turned, in float64."""
    x = as_float64(x)
    f = np.asarray(inv_freq.detach().cpu() if hasattr(inv_freq, "detach") else inv_freq, dtype=np.float64)
    angle = as_int64(positions)[:, None].astype(np.float64) * f[None, :]
    turn = factor * np.exp((-1j if inverse else 1j) * angle)[:, None, :]
    d0, d1 = pair_dims(2 * len(f), offset, interleaved)
    z = (x[..., d0] + 1j * x[..., d1]) * turn
    y = x.copy()
    y[..., d0], y[..., d1] = z.real, z.imag
    return y


def rotate_f32(x, positions, table, *, interleaved: bool = False, offset: int = 0) -> np.ndarray:
    """x turned in float32 by the rows of table float32 [n_positions, rot / 2, 2]."""
    x = as_float64(x).astype(np.float32)
    cs = np.asarray(table, dtype=np.float32)[as_int64(positions)]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    d0, d1 = pair_dims(2 * cs.shape[1], offset, interleaved)
    a, b = x[..., d0], x[..., d1]
    y = x.copy()
    y[..., d0] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
    y[..., d1] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return y
