"""Bounded waits of cross attention and shared prefixes, exercised without a GPU fault.

The library's test hook makes CTA 0 skip the copy of one tile of K, so the wait for that tile, and after it those of the
CTA's other warps, can only end by running out.  The call must return with FP8MLA_DEV_WAIT_TIMEOUT recorded, rows of other
CTAs' items as they are, and the next call, with the hook off, reproduces the run before it.
"""

import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from tests import ragged_inputs as inputs
from tests.test_cross_gpu import _call as cross
from tests.test_shared_gpu import _call as shared

pytestmark = pytest.mark.gpu

LIMIT_NS = 20_000_000  # 20 ms: longer than any of these calls, short enough for a fast test


def _runs_out(call, fault):
    fm.last_device_error()
    before = call()
    assert fm.last_device_error() == 0
    try:
        fm.set_wait_test(fault, LIMIT_NS)
        during = call()
        code = fm.last_device_error()
    finally:
        fm.set_wait_test(0, 0)
    assert code == fm.DEV_WAIT_TIMEOUT
    after = call()
    assert fm.last_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    return before, during


def _cross_call(seed, bs, tokens, keys, hd, rows):
    pool = inputs.Pool(seed, [[keys] * bs], 1, hd, 64, rows)
    q = pool.queries(bs * tokens, 1)
    starts = list(range(0, bs * tokens + 1, tokens))
    return lambda: cross(pool, q, [keys] * bs, starts)


# few rows, one stream, a pair; an item a CTA, one in many shares
@pytest.mark.parametrize("hd,rows", [(64, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("bs,tokens,keys,fault", [(1, 3, 300, 1), (1, 3, 300, 3), (152, 60, 600, 1), (152, 60, 600, 3),
                                                  (152, 150, 600, 1), (152, 150, 600, 3), (1, 3, 60000, 1),
                                                  (1, 600, 20000, 1)])
def test_cross(hd, rows, bs, tokens, keys, fault):
    _runs_out(_cross_call(31, bs, tokens, keys, hd, rows), fault)


def test_several_items_and_other_ctas():
    """CTA 0 has many items; it gives up in the middle, the others' rows are right."""
    n = 1500
    before, during = _runs_out(_cross_call(32, n, 1, 300, 64, True), 8)
    wrong = torch.nonzero(~(before[0] == during[0]).all(-1).all(-1))
    assert wrong.numel() > 0 and int(wrong.max()) < n // 50  # the first share's items


@pytest.mark.parametrize("q_len,hd", [(1, 64), (3, 128)])
@pytest.mark.parametrize("fault", [1, 2])
def test_shared(q_len, hd, fault):
    lens = [500, 7, 130]
    pool, q, m, s, want = inputs.shared_case(33, [900], [0, 2], lens, 1, 2, hd, 16, hd == 64, q_len=q_len, sinks=True)
    before, _ = _runs_out(lambda: shared(pool, q, [900], [0, 2], lens, m, s), fault)
    assert inputs.within(*before, want, 1400) is None


def test_items_longer_than_the_limit():
    """A warp that tells items waits for whole ones: their length is no sign of a hang.  Each CTA has one of 2^26 keys (about
    half a second, the limit is 20 ms and 65536 polls, a quarter of a second) and some of a few keys."""
    dev, sms = torch.device("cuda"), torch.cuda.get_device_properties(0).multi_processor_count
    gen = torch.Generator(device=dev).manual_seed(34)
    k, v = (torch.randn(8, 1, 256, 64, generator=gen, device=dev).to(torch.float8_e4m3fn) for _ in range(2))
    group = torch.tensor([256, 1, 1, 1, 1], dtype=torch.int32, device=dev).repeat(sms)
    lens = torch.where(group == 256, 1 << 26, 20).to(torch.int32)
    starts = torch.cat((torch.zeros(1, dtype=torch.int32, device=dev), group.cumsum(0, dtype=torch.int32)))
    q = torch.randn(int(starts[-1]), 1, 64, generator=gen, device=dev).to(torch.bfloat16)
    table = (torch.arange((1 << 26) // 256, device=dev, dtype=torch.int32) % 8).expand(5 * sms, -1).contiguous()
    one = torch.ones(1, device=dev)
    fm.last_device_error()
    try:
        fm.set_wait_test(0, LIMIT_NS)
        out, lse = fm.paged_cross_attention(q, k, v, table, lens, one, one, q_starts=starts)
        assert fm.last_device_error() == 0
    finally:
        fm.set_wait_test(0, 0)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    short = torch.repeat_interleave(group == 1, group.long())
    want = fm.paged_cross_attention(q[short], k, v, table[:4 * sms, :1].contiguous(), lens[group == 1], one, one)
    assert torch.equal(out[short], want[0]) and torch.equal(lse[short], want[1])
