"""Pins of the rotary and 4-bit oracles, and of the host-side frequencies."""

import math

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from oracle import fp4
from oracle.rotary import rotate, rotate_f32


def test_e2m1_values_and_ties():
    assert [fp4.e2m1_value(c) for c in range(8)] == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert [fp4.e2m1_value(8 + c) for c in range(1, 8)] == [-0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
    # midpoints go to the even code: 0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0
    mid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert fp4.e2m1_encode(mid).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert fp4.e2m1_encode(np.nextafter(mid, 9)).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert fp4.e2m1_encode(np.nextafter(mid, 0)).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert fp4.e2m1_encode([7.0, -100.0, -0.1]).tolist() == [7, 15, 8]


def test_fp4_round_trip_of_representable_rows():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, (5, 4, 16))
    codes[..., 0] = 7  # every block holds the largest value, so its scale is the one it was made with
    s8 = np.array([1.0, 0.5, 448.0, 2.0 ** -6])
    x = (fp4.E2M1_TABLE[codes] * s8[None, :, None]).reshape(5, 64)
    packed, scales = fp4.quantise(x, 1.0)
    assert np.array_equal(fp4.dequantise(packed, scales, 1.0), x)
    # low nibble = even dimension
    assert packed[0, 0] & 15 == 7


def test_fp4_zero_and_tiny_blocks():
    packed, s8 = fp4.quantise(np.zeros((1, 32)), 0.25)
    assert not packed.any() and not s8.any()
    x = np.zeros((1, 32))
    x[0, 3] = -1e-6  # amax / 6 rounds to a zero scale
    packed, s8 = fp4.quantise(x, 1.0)
    assert not packed.any() and not s8.any()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_the_distance(interleaved):
    rng = np.random.default_rng(1)
    f, _ = fm.rotary_frequencies(32)
    q, k = rng.standard_normal((2, 1, 1, 48))
    at = lambda x, p: rotate(x, [p], f, interleaved=interleaved, offset=8)  # noqa: E731
    assert np.allclose(np.linalg.norm(at(q, 12345)), np.linalg.norm(q))
    assert np.array_equal(at(q, 77)[..., :8], q[..., :8]) and np.array_equal(at(q, 77)[..., 40:], q[..., 40:])
    assert np.allclose(np.sum(at(q, 900) * at(k, 850)), np.sum(at(q, 50) * at(k, 0)))
    assert np.allclose(rotate(at(q, 31), [31], f, interleaved=interleaved, offset=8, inverse=True), q)
    assert np.array_equal(at(q, 0), q)


def test_rotation_of_a_quarter_turn_by_hand():
    f = np.array([math.pi / 2, math.pi])
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    # half layout: pairs (1, 3) by 90 degrees, (2, 4) by 180
    assert np.allclose(rotate(x, [1], f), [[[-3.0, -2.0, 1.0, -4.0]]])
    # interleaved: pairs (1, 2) and (3, 4)
    assert np.allclose(rotate(x, [1], f, interleaved=True, factor=2.0), [[[-4.0, 2.0, -6.0, -8.0]]])


def test_float32_rotation_is_near_the_definition():
    rng = np.random.default_rng(2)
    f, _ = fm.rotary_frequencies(64)
    pos = np.array([0, 5, 4095])
    angle = np.arange(4096)[:, None] * f.numpy()
    table = np.stack((np.cos(angle), np.sin(angle)), -1).astype(np.float32)
    x = rng.standard_normal((3, 2, 64)).astype(np.float32)
    # two products of a table entry (each within 2^-24) and a sum
    bound = 4 * 2.0 ** -24 * (np.abs(x[..., :32]) + np.abs(x[..., 32:]))
    err = np.abs(rotate_f32(x, pos, table) - rotate(x, pos, f))
    assert np.all(err <= np.concatenate((bound, bound), -1))


def test_frequencies_of_each_scaling():
    f, a = fm.rotary_frequencies(8, 10000.0)
    assert a == 1.0 and np.allclose(f, [1.0, 0.1, 0.01, 0.001])
    g, a = fm.rotary_frequencies(8, 10000.0, dict(type="linear", factor=4))
    assert a == 1.0 and np.allclose(g * 4, f)
    g, _ = fm.rotary_frequencies(8, 10000.0, dict(type="ntk", factor=4))
    assert np.allclose(g[0], 1.0) and np.allclose(g[-1], f[-1] / 4)  # the slowest pair is stretched by the factor
    g, a = fm.rotary_frequencies(8, 10000.0, dict(type="bands", factor=8, trained=1000))
    # turns over 1000 positions: 159, 15.9, 1.59, 0.159
    keep = (10 / (2 * math.pi) - 1) / 3
    assert a == 1.0 and np.allclose(g, [1.0, 0.1, 0.01 * keep + 0.01 / 8 * (1 - keep), 0.001 / 8])
    g, a = fm.rotary_frequencies(64, 10000.0, dict(type="yarn", factor=16, trained=4096))
    base, _ = fm.rotary_frequencies(64)
    assert np.isclose(a, 0.1 * math.log(16) + 1) and np.allclose(g[0], base[0]) and np.allclose(g[-1], base[-1] / 16)
    assert torch.all(g <= base * (1 + 1e-12)) and torch.all(g >= base / 16 * (1 - 1e-12))
    g, a = fm.rotary_frequencies(4, 100.0, dict(type="factors", factors=[1.0, 2.0], attention=1.5))
    assert a == 1.5 and np.allclose(g, [1.0, 0.05])


@pytest.mark.parametrize("bad", [dict(type="other"), dict(factor=2), dict(type="linear"), dict(type="linear", factor=0),
                                 dict(type="linear", factor=2, trained=5), dict(type="yarn", factor=2),
                                 dict(type="bands", factor=2, trained=8, low=4, high=4),
                                 dict(type="factors", factors=[1.0]), dict(type="factors", factors=[1, 1, 1, 0])])
def test_frequencies_refuse(bad):
    with pytest.raises(ValueError):
        fm.rotary_frequencies(8, 10000.0, bad)


def test_frequencies_refuse_sizes():
    for rot, theta in ((7, 1e4), (0, 1e4), (8, 0.0), (8, math.inf)):
        with pytest.raises(ValueError):
            fm.rotary_frequencies(rot, theta)
