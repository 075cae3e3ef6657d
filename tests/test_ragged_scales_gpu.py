"""Cross attention and shared prefixes with V row scales far from one, against the float64 oracle.

Tolerances: those of tests/ragged_inputs.py, and beside them, before any run: a weight carries 2^(log2 of its V scale),
whose approximate logarithm is off by 2^-22 of its size (150 at most) as is float32's sum with the score; f16's spacing
below its normal numbers is 2^-24 where the largest weight times V scale is 2^7 or more, which is no more than the largest
V scale, so it is keys * 2^-32 * 448 of that; bf16's spacing below its normal numbers is 2^-133, and values that small pass
float32 numbers whose spacing is 2^-149 for each of the partial sums.
"""

import numpy as np
import pytest
import torch

from tests import ragged_inputs as inputs
from tests.test_cross_gpu import _call as cross
from tests.test_shared_gpu import _call as shared

pytestmark = pytest.mark.gpu


def _powers(rng, pattern, keys):
    """What the V scales of a sequence's keys are multiplied by."""
    j = np.arange(keys)
    if pattern == "one":  # a row of the smallest scales among ordinary ones
        x = np.zeros(keys)
        x[rng.integers(keys)] = -140
    elif pattern == "mixed":
        x = rng.uniform(-140, 20, keys)
    elif pattern == "wide":
        x = rng.uniform(-50, 50, keys)
    elif pattern == "rising":  # by tile
        x = np.minimum(-140 + 40.0 * (j // 128), 60)
    elif pattern == "falling":
        x = np.maximum(30 - 50.0 * (j // 128), -140)
    elif pattern in ("zeros", "zeros first"):
        x = np.where(rng.random(keys) < 0.3 if pattern == "zeros" else j < 140, -np.inf, 0)
    else:
        x = np.full(keys, float(pattern))
    return np.exp2(x)


PATTERNS = ["one", "mixed", "wide", "rising", "falling", "zeros", "zeros first", "-150", "-135", "-115", "-60", "45", "90"]


def _rescale(pool, table, lens, pattern):
    for b, n in enumerate(lens):
        if n == 0:
            continue
        f = _powers(pool.rng, pattern, int(n))
        j = np.arange(int(n))
        at = table[b][j // pool.page], slice(None), j % pool.page
        pool.scale[1][at] = (pool.scale[1][at].astype(np.float64) * f[:, None]).astype(np.float32)


def _within(got, want, keys, pool):
    sv = pool.scale[1]
    top = np.nanmax(sv)
    used = sv[np.isfinite(sv) & (sv > 0)]
    far = np.abs(np.log2(used.astype(np.float64))).max() if used.size else 0.0
    out, lse, pv, most, size = want
    tol_out, tol_lse = inputs.tolerance((out, lse, pv, np.zeros_like(most), size), keys)
    tol_out = tol_out + 2.0 ** -21 * far * pv + keys * 2.0 ** -32 * 448.0 * float(top) + 2.0 ** -134 + keys * 2.0 ** -149
    tol_lse = tol_lse + 2.0 ** -21 * far
    g_out = got[0].double().cpu().numpy().reshape(out.shape)
    g_lse = got[1].double().cpu().numpy().reshape(lse.shape)
    assert np.array_equal(g_lse == -np.inf, lse == -np.inf)
    some = lse > -np.inf
    bad = ~(np.abs(g_lse[some] - lse[some]) <= tol_lse[some])
    assert not bad.any(), f"lse: {bad.sum()} of {bad.size}, {g_lse[some][bad][:4]} for {lse[some][bad][:4]}"
    bad = ~(np.abs(g_out - out) <= tol_out)
    assert not bad.any(), f"out: {bad.sum()} of {bad.size}, {g_out[bad][:4]} for {out[bad][:4]}"


# few rows, one stream, a pair of streams, all of them; items that are cut
@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q_lens,lens,group", [([3], [300], 2), ([40], [300], 2), ([150], [300], 1),
                                               ([290, 2, 30], [270, 20, 700], 1), ([2, 50, 130], [3000, 2500, 2000], 1)])
def test_cross(pattern, hd, q_lens, lens, group):
    pool, q, starts, _ = inputs.cross_case(3, q_lens, lens, 1, group, hd, 16, True)
    _rescale(pool, pool.tables[0], lens, pattern)
    want = inputs.ragged.cross(q, *pool.cache, pool.tables[0], lens, *pool.scale, pool.softmax_scale, starts)
    _within(cross(pool, q, lens, starts), want, max(lens), pool)


@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("hd,q_len", [(64, 1), (128, 3)])
def test_shared(pattern, hd, q_len):
    """Each half with its own scales: the batch's first prefix and own keys as the pattern, the others as they are."""
    lens, prefixes, first = [200, 3, 0, 600], [1500, 90], [0, 2, 4]
    pool, q, m, s, _ = inputs.shared_case(4, prefixes, first, lens, 2, 2, hd, 32, True, q_len=q_len, sinks=True)
    _rescale(pool, pool.tables[0], prefixes[:1], pattern)
    _rescale(pool, pool.tables[1], lens[:3], pattern)
    want = inputs.ragged.shared(q, *pool.cache, pool.tables[0], prefixes, first, pool.tables[1], lens, *pool.scale,
                                pool.softmax_scale, m, s)
    _within(shared(pool, q, prefixes, first, lens, m, s), want, 2200, pool)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("tokens", [2, 40, 150])
def test_a_small_row_that_has_the_weight(hd, tokens):
    """Scores that lead by hundreds on rows of small scales: their values come back, not those of rows of large ones."""
    lens = [400]
    pool, q, starts, _ = inputs.cross_case(5, [tokens], lens, 1, 1, hd, 16, True)
    q[..., 0] = 64.0
    j = np.arange(400)
    at = pool.tables[0][0][j // 16], 0, j % 16
    pool.cache[0][(*at, 0)] = inputs.e4m3_encode(np.where(j % 7 == 3, 0.0, -448.0))
    pool.scale[0][at] = 2.0 ** -4
    pool.scale[1][at] = np.where(j % 7 == 3, 2.0 ** -100, 2.0 ** 10).astype(np.float32)
    want = inputs.ragged.cross(q, *pool.cache, pool.tables[0], lens, *pool.scale, pool.softmax_scale, starts)
    assert np.abs(want[0]).max() < 2.0 ** -90
    out, lse = cross(pool, q, lens, starts)
    err = 2.0 ** -15 * want[4] + 2.0 ** -14 + 2.0 ** -10
    assert np.all(np.abs(lse.double().cpu().numpy() - want[1]) <= err)
    assert np.all(np.abs(out.double().cpu().numpy() - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 2 * err[..., None] * want[2])
