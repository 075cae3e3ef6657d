"""Decode over the 4-bit cache where scores are so large that float32 holds them in steps of many units.

Tolerances, before any run.  A score is off by no more than e = (hd + 8) 2^-23 S, S = scale max_j sum_d |q_d k_jd|:
the sum's head_dim roundings, the factor's and the product's, and two references' of a merge.  Rows are taken whose
best key leads by 2 e + 40 nats, so that the others weigh at most e^-40 together with the error, and the row is that
key's V: its weight and the sum hold the same weight, rounded to f16 in the one (2^-11) and not in the other, with
2^-20 for the approximate functions, and bf16's rounding is 2^-8 of the value.  A key that weighs nothing adds at most
keys * 2^-32 of the largest |v| (f16's smallest step beside the largest weight, 2^7).  The LSE is off by e, the
rounding to float32 and 2^-21.
"""

import math

import numpy as np
import pytest
import torch

from oracle import fp4
from oracle.attention import spec_visible
from tests.test_gqa_fp4_gpu import Inputs

SIZES = (0, 14, 19, 21, 23, 25, 27, 28, 29, 30, 33, 40, 64, 100)  # log2 of the queries' scale, dealt to heads in turn


def _scaled(x, first=0):
    """x with head h's queries 2^SIZES[h + first] times as large."""
    q = x.q.double()
    for h in range(q.shape[2]):
        q[:, :, h] *= 2.0 ** SIZES[(h + first) % len(SIZES)]
    x.q = q.to(torch.bfloat16)
    return x


def _led(x, window, rows):
    """{(b, i, h): (e, lead)} of the rows: the scores' error and by how much the best key leads, in nats."""
    found = {}
    q, mask = x.q.double().numpy(), None if x.mask is None else x.mask.numpy()
    page, group = x.codes[0].shape[2], x.q.shape[2] // x.codes[0].shape[1]
    for b, h in rows:
        n = int(x.lens[b])
        pages, kvh = x.bt[b, :-(-n // page)], h // group
        k = np.concatenate([np.zeros((0, x.hd))] + [fp4.dequantise(x.codes[0][p, kvh], x.s8[0][p, kvh], x.scale[0])
                                                    for p in pages])[:n]
        for i in range(q.shape[1]):
            vis = spec_visible(n, q.shape[1], i, None if mask is None else mask[b, i].astype(np.int64), window)
            s = np.sort((k[vis] @ q[b, i, h]) * x.softmax_scale)[::-1]
            big = (np.abs(k[vis]) @ np.abs(q[b, i, h])).max() * x.softmax_scale if len(s) else 0.0
            if x.sinks is not None:
                s = np.sort(np.append(s, float(x.sinks[h])))[::-1]
            found[b, i, h] = (x.hd + 8) * 2.0 ** -23 * big, s[0] - s[1] if len(s) > 1 else math.inf
    return found


def _check(x, out, lse, window=0, rows=None):
    if rows is None:
        rows = [(b, h) for b in range(len(x.lens)) for h in range(x.q.shape[2])]
    want, want_lse, weight = x.want(window, rows)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    vmax = 6 * 448 * x.scale[1]
    taken = 0
    for (b, i, h), (e, lead) in _led(x, window, rows).items():
        o, l, a = want[b, i, h], want_lse[b, i, h], weight[b, i, h]
        if np.isneginf(l):
            assert np.isneginf(got_lse[b, i, h]) and np.all(got[b, i, h] == 0)
            continue
        if abs(l) < 1e38:
            assert abs(got_lse[b, i, h] - l) <= e + 2.0 ** -21 + 2.0 ** -22 * abs(l), (b, i, h, got_lse[b, i, h], l)
        if lead < 2 * e + 40:
            continue
        taken += 1
        tol = 2.0 ** -8 * np.abs(o) + (1 + 2.0 ** -8) * (a * (2.0 ** -11 + 2.0 ** -20) +
                                                         int(x.lens.max()) * 2.0 ** -32 * vmax)
        assert np.all(np.abs(got[b, i, h] - o) <= tol), (b, i, h, np.abs(got[b, i, h] - o).max(), tol.max())
    return taken


def test_the_rows_taken_are_most_of_them():
    """Of random keys the best one leads by enough at nearly every size but the first."""
    x = _scaled(Inputs(1, [300, 5], 1, 14, 128, 16))
    led = [lead >= 2 * e + 40 for e, lead in _led(x, 0, [(b, h) for b in range(2) for h in range(14)]).values()]
    assert sum(led) >= 23


@pytest.mark.gpu
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("group", [4, 14])
def test_short_and_asked_for_shards(hd, group):
    x = _scaled(Inputs(hd + group, [300, 0, 1, 16, 17, 900, 129], 2, group, hd, 16))
    for splits in (0, 1, 5):  # clusters and wide CTAs, one CTA, shards
        assert _check(x, *x.run(num_splits=splits)) >= 0.7 * 12 * group


@pytest.mark.gpu
def test_one_key_each_weighs_one():
    """A context of one key returns its V whatever the score, of either sign."""
    x = _scaled(Inputs(2, [1] * 40, 2, 14, 128, 16))
    for splits in (0, 1):
        assert _check(x, *x.run(num_splits=splits)) == 40 * 28


@pytest.mark.gpu
def test_pieces_and_many_short_sequences():
    x = _scaled(Inputs(3, [9001], 1, 14, 128, 16))
    assert _check(x, *x.run()) >= 10
    x = _scaled(Inputs(4, [4000, 3000, 1], 1, 7, 64, 64), first=7)
    assert _check(x, *x.run()) >= 18
    x = _scaled(Inputs(5, [100] * 240, 2, 7, 64, 16), first=7)  # more sequences than CTAs fit
    assert _check(x, *x.run(), rows=[(b, h) for b in (0, 7, 239) for h in range(14)]) >= 36


@pytest.mark.gpu
@pytest.mark.parametrize("mask,window,sinks,group", [(True, 0, False, 4), (False, 37, True, 2), (True, 100, True, 7)])
def test_blocks_windows_and_sinks(mask, window, sinks, group):
    for first in (3, 9):
        x = _scaled(Inputs(60 + group, [700, 3, 0, 48, 129], 2, group, 128, 16, 4, mask, sinks), first)
        for splits in (0, 1, 3):
            _check(x, *x.run(window=window, num_splits=splits), window=window)


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_that_rise_or_fall_along_the_keys(sign):
    """The reference moves with nearly every page, or never again."""
    x = _scaled(Inputs(7, [600, 500], 1, 4, 128, 16), first=6)
    k = fp4.dequantise(x.codes[0], np.where(x.s8[0] & 0x7F == 0x7F, 0, x.s8[0]))[:, 0]
    best = (k @ x.q[0, 0, 0].double().numpy()).max(-1)
    whole = x.bt[0, :37]
    x.bt[0, :37] = whole[np.argsort(sign * best[whole])]
    for splits in (0, 1, 2):
        assert _check(x, *x.run(num_splits=splits)) >= 7
