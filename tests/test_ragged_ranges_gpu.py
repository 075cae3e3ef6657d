"""Cross attention whose token ranges do not fit: they count as empty, in outputs that the call makes too."""

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from tests import ragged_inputs as inputs
from tests.test_cross_gpu import _call

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _used_memory(q):
    """Leaves blocks of the outputs' sizes to the allocator, which hold other numbers."""
    blocks = [torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(8)]
    blocks += [torch.full(q.shape[:2], 5.0, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("hd,group", [(64, 2), (128, 1)])
@pytest.mark.parametrize("starts", [
    [0, 4, 8, 13],                # the last range passes the tokens
    [0, 100, 6, 12],              # a range that does, the next one falls
    [0, 8, 4, 4],                 # falling: the first range is kept, the tokens behind it have none
    [-3, 2, 5, 12],               # in front of the tokens
    [-5, -2, -1, -1], [20, 30, 40, 50], [7, 3, 2, 1], [0, 5, 2147483647, 12], [-2147483648, 0, 3, 9]])
def test_ranges_that_do_not_fit(starts, hd, group):
    lens, n = [40, 33, 20], 12
    pool, q, _, _ = inputs.cross_case(21, [4, 4, 4], lens, 1, group, hd, 16, False)
    kept = [max(a, 0) if 0 <= a <= b <= n else None for a, b in zip(starts, starts[1:])]
    want = [np.full(x.shape, -np.inf) if i == 1 else np.zeros(x.shape) for i, x in
            enumerate(inputs.ragged.cross(q, *pool.cache, pool.tables[0], lens, *pool.scale, pool.softmax_scale))]
    for b, first in enumerate(kept):
        if first is not None:
            at = slice(starts[b], starts[b + 1])
            one = inputs.ragged.cross(q[at], *pool.cache, pool.tables[0][b:b + 1], lens[b:b + 1], *pool.scale,
                                      pool.softmax_scale, [0, starts[b + 1] - starts[b]])
            for w, x in zip(want, one):
                w[at] = x
    fm.last_device_error()
    _used_memory(q)
    out, lse = _call(pool, q, lens, starts)
    assert fm.last_device_error() == fm.DEV_BAD_SEQLEN
    wrong = inputs.within(out, lse, want, 40)
    assert wrong is None, wrong


def test_many_ranges_one_of_which_does_not_fit():
    rng = np.random.default_rng(5)
    q_lens, lens = rng.integers(0, 3, 900).tolist(), rng.integers(0, 30, 900).tolist()
    pool, q, starts, want = inputs.cross_case(22, q_lens, lens, 1, 1, 64, 16, False, pad=(3, 40))
    bad = int(np.flatnonzero(np.asarray(q_lens) > 0)[450])
    starts = starts.copy()
    starts[bad + 1:] += 2 * len(q)  # from here on no range fits
    for i, w in enumerate(want):
        w[starts[bad]:] = -np.inf if i == 1 else 0
    _used_memory(q)
    out, lse = _call(pool, q, lens, starts)
    assert fm.last_device_error() == fm.DEV_BAD_SEQLEN
    wrong = inputs.within(out, lse, want, 30)
    assert wrong is None, wrong
    # given outputs keep what they held there
    out, lse = torch.full_like(q.to(DEV), 7.0), torch.full(q.shape[:2], 5.0, device=DEV)
    _call(pool, q, lens, starts, out=out, lse=lse)
    assert fm.last_device_error() == fm.DEV_BAD_SEQLEN
    at = int(starts[bad])
    assert bool((out[at:] == 7).all()) and bool((lse[at:] == 5).all()) and bool((out[:3] == 7).all())


def test_many_tokens_between_ranges():
    """Ranges of thousands of tokens with gaps between them that falling and far starts leave."""
    n = 20000
    pool = inputs.Pool(23, [[40] * 8], 1, 64, 16, False)
    k, v, table, ks, vs = pool.device(DEV)
    q = pool.queries(n, 1).to(DEV)
    starts = [0, 9001, 9001, 30000, 12000, 16999, 16999, 19998, 20001]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    lens = i32([40, 3, 40, 40, 33, 40, 7, 40])
    want, want_lse = torch.zeros_like(q), torch.full((n, 1), -float("inf"), device=DEV)
    for b, (lo, hi) in enumerate(zip(starts, starts[1:])):
        if lo < hi <= n:
            want[lo:hi], want_lse[lo:hi] = fm.paged_cross_attention(
                q[lo:hi], k, v, table[b:b + 1], lens[b:b + 1], ks, vs, q_starts=i32([0, hi - lo]))
    fm.last_device_error()
    _used_memory(q)
    out, lse = fm.paged_cross_attention(q, k, v, table, lens, ks, vs, q_starts=i32(starts))
    assert fm.last_device_error() == fm.DEV_BAD_SEQLEN
    gaps = torch.zeros(n, dtype=torch.bool, device=DEV)
    gaps[9001:12000], gaps[19998:] = True, True
    assert bool((out[gaps] == 0).all()) and bool((lse[gaps] == -float("inf")).all())
    assert bool(torch.isfinite(lse[~gaps]).all())
    # the same rows from items that are cut elsewhere: either rounds to bf16 (2^-8) and weighs in f16 (2^-11 of |v|)
    most = float(v.float().nan_to_num().abs().max()) * float(vs)  # (NaN where no key is)
    assert bool(((out.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -10 * most).all())
    assert bool(((lse - want_lse).abs()[~gaps] <= 2.0 ** -16 * 40).all())
