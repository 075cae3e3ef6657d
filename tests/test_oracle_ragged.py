"""The oracle of cross attention, shared prefixes and merges, held to the other oracles, and the tolerance of the GPU
tests, which wrong results miss."""

import numpy as np
import pytest
import torch

from oracle import attention, ragged
from tests import ragged_inputs as inputs


@pytest.mark.parametrize("rows", [False, True])
def test_cross_of_single_tokens_is_a_decode(rows):
    lens = [1, 40, 0, 17]
    pool, q, _, want = inputs.cross_case(1, [1] * 4, lens, 2, 3, 64, 16, rows)
    scales = pool.scale if rows else [float(s[0]) for s in pool.scale]
    out, lse = attention.gqa_decode_ext(q.unsqueeze(1), *pool.cache, pool.tables[0], lens, *scales,
                                        pool.softmax_scale)[:2]
    assert np.allclose(want[0], out[:, 0], rtol=0, atol=1e-12) and np.allclose(want[1], lse[:, 0], rtol=0, atol=1e-12)


@pytest.mark.parametrize("q_len,mask,sinks", [(1, False, False), (3, False, True), (4, True, False), (2, True, True)])
def test_shared_is_a_decode_over_both_tables(q_len, mask, sinks):
    """Prefixes of whole pages: the tables of a decode that holds them per sequence are the two tables in a row."""
    prefix_lens, starts, lens = [32, 48], [1, 3, 4], [7, 20, 4, 33, 16]
    pool, q, m, s, want = inputs.shared_case(2, prefix_lens, starts, lens, 2, 2, 64, 16, False, q_len, mask, sinks)
    table, total = np.zeros((5, 8), np.int32), []
    for b in range(5):
        g = next((g for g in range(2) if starts[g] <= b < starts[g + 1]), None)
        front = 0 if g is None else prefix_lens[g] // 16
        if front:
            table[b, :front] = pool.tables[0][g, :front]
        own = -(-lens[b] // 16)
        table[b, front:front + own] = pool.tables[1][b, :own]
        total.append(front * 16 + lens[b])
    out, lse = attention.gqa_decode_ext(q, *pool.cache, table, total, *[float(x[0]) for x in pool.scale],
                                        pool.softmax_scale, m, 0, s)[:2]
    assert np.allclose(want[0], out.reshape(want[0].shape), rtol=0, atol=1e-12)
    assert np.allclose(want[1], lse.reshape(want[1].shape), rtol=0, atol=1e-12)


def test_merge_of_parts_is_the_whole():
    rng = np.random.default_rng(3)
    k, v, q = rng.standard_normal((30, 8)), rng.standard_normal((30, 8)), rng.standard_normal(8)
    whole = ragged.attend(q, k, v, 0.3)
    cuts = [0, 4, 4, 21, 30]  # one part without keys
    parts = [ragged.attend(q, k[a:b], v[a:b], 0.3) for a, b in zip(cuts, cuts[1:])]
    out, lse = ragged.merge([p[0][None, None] for p in parts], [np.array([[p[1]]]) for p in parts])
    assert np.allclose(out[0, 0], whole[0], atol=1e-14) and abs(lse[0, 0] - whole[1]) < 1e-14
    out, lse = ragged.merge([np.full((1, 1, 2), np.nan)] * 2, [np.full((1, 1), -np.inf)] * 2)
    assert np.all(out == 0) and lse[0, 0] == -np.inf
    triple = attention.merge_partials([attention.partial_attention(k[a:b] @ q * 0.3, v[a:b]) for a, b in zip(cuts, cuts[1:])])
    assert np.allclose(triple[0], whole[0], atol=1e-14) and abs(triple[1] - whole[1]) < 1e-14


def _rounded(want):
    return torch.from_numpy(want[0]).to(torch.bfloat16), torch.from_numpy(want[1]).float()


@pytest.mark.parametrize("rows", [False, True])
def test_the_tolerance_tells_wrong_results(rows):
    q_lens, kv_lens, keys = [3, 5], [150, 90], 150
    pool, q, starts, want = inputs.cross_case(4, q_lens, kv_lens, 2, 2, 64, 16, rows)
    assert inputs.within(*_rounded(want), want, keys) is None

    def other(table=pool.tables[0], lens=kv_lens, cache=pool.cache, scale=pool.scale, at=starts, x=q):
        got = ragged.cross(x, *cache, table, lens, *scale, pool.softmax_scale, at)
        return inputs.within(*_rounded(got), want, keys)

    assert other(lens=[149, 90]) and other(lens=[150, 89])                   # a key too few
    assert other(at=np.array([0, 4, 8])) and other(x=q.flip(1))              # tokens, heads exchanged
    swapped = pool.tables[0].copy()
    swapped[0, [2, 3]] = swapped[0, [3, 2]]
    if rows:  # an exchanged page changes nothing where all keys are seen: the scales alone give it away
        shifted = [np.roll(np.nan_to_num(s, nan=1.0), 1, axis=2) for s in pool.scale]
        assert other(scale=shifted)
    assert other(table=np.where(swapped == swapped[0, 2], swapped[0, 3], swapped))  # a page twice
    one = [c.copy() for c in pool.cache]
    one[1][pool.tables[0][0, 1], 0, 3, 5] ^= 0x20                            # a value's exponent
    assert other(cache=one)
    third = want[0].copy()
    third[0, 0] *= 1 + 2.0 ** -6
    assert inputs.within(torch.from_numpy(third), torch.from_numpy(want[1]), want, keys)


def test_the_tolerance_tells_a_wrong_block():
    pool, q, m, s, want = inputs.shared_case(5, [40], [0, 2], [9, 12, 30], 1, 2, 64, 16, False, 3, True, True)
    assert inputs.within(*_rounded(want), want, 70) is None
    args = (q, *pool.cache, pool.tables[0], [40], [0, 2], pool.tables[1], [9, 12, 30], *pool.scale, pool.softmax_scale)
    for wrong in (dict(mask=1 - m, sinks=s), dict(mask=None, sinks=s), dict(mask=m, sinks=None), dict(mask=m, sinks=s[::-1])):
        assert inputs.within(*_rounded(ragged.shared(*args, **wrong)), want, 70)
    assert inputs.within(*_rounded(ragged.shared(*args[:5], [0, 3], *args[6:], mask=m, sinks=s)), want, 70)
