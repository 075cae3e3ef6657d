"""Decode behind shared prefixes on the GPU against the float64 oracle (tolerances: tests/ragged_inputs.py)."""

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from tests import ragged_inputs as inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).to(DEV)


def _call(pool, q, prefix_lens, prefix_starts, lens, mask=None, sinks=None, **kw):
    k, v, ptable, table, ks, vs = pool.device(DEV)
    out, lse = fm.paged_gqa_decode_shared(
        q.to(DEV) if not q.is_cuda else q, k, v, ptable, _i32(prefix_lens), _i32(prefix_starts), table, _i32(lens), ks, vs,
        softmax_scale=pool.softmax_scale, spec_mask=None if mask is None else torch.from_numpy(mask).to(DEV),
        sinks=None if sinks is None else torch.from_numpy(sinks).to(DEV), **kw)
    torch.cuda.synchronize()
    return out, lse


def _check(seed, prefix_lens, starts, lens, h_kv, group, hd, page, rows, **kw):
    pool, q, m, s, want = inputs.shared_case(seed, prefix_lens, starts, lens, h_kv, group, hd, page, rows, **kw)
    out, lse = _call(pool, q, prefix_lens, starts, lens, m, s)
    wrong = inputs.within(out, lse, want, max([0, *prefix_lens]) + max(lens) + 1)
    assert wrong is None, wrong
    assert fm.last_device_error() == 0


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("prefix_lens,starts,lens,h_kv,group,q_len", [
    ([1], [0, 1], [1], 1, 1, 1),
    ([200], [0, 4], [5, 129, 1, 64], 2, 4, 1),
    ([0], [0, 2], [3, 0], 1, 3, 1),                      # an empty prefix; a row without any key
    ([300, 0, 77], [1, 3, 3, 5], [0, 0, 40, 17, 130, 9], 1, 2, 1),  # no prefix, nothing of its own, a prefix of none
    ([150], [0, 70], [3] * 70, 1, 4, 1),                 # more rows than an item
    ([129, 40], [0, 2, 5], [4, 90, 2, 3, 140], 2, 2, 4),  # blocks; shorter than the block
    ([260], [0, 6], [1, 2, 33, 8, 5, 0], 1, 7, 2),
    ([64], [0, 3], [40, 41, 32], 1, 1, 32)])
def test_shapes(prefix_lens, starts, lens, h_kv, group, q_len, hd, rows):
    _check(1, prefix_lens, starts, lens, h_kv, group, hd, 16, rows, q_len=q_len)


@pytest.mark.parametrize("q_len,mask,sinks", [(1, False, True), (1, True, False), (4, True, False), (4, True, True),
                                              (8, False, True)])
def test_masks_and_sinks(q_len, mask, sinks):
    """Random masks: rows that see nothing of their block, and (no prefix, no other key) nothing at all."""
    _check(2, [100], [2, 5], [q_len, 0, 50, q_len, 9, q_len + 1], 2, 2, 128, 32, True, q_len=q_len, mask=mask, sinks=sinks)


def test_a_mask_that_hides_everything():
    pool, q, _, _, _ = inputs.shared_case(3, [0], [0, 1], [2, 2], 1, 2, 64, 16, False, 2)
    m = np.zeros((2, 2, 2), np.uint8)
    for s in (None, np.array([0.5, -3.0], np.float32)):
        want = inputs.ragged.shared(q, *pool.cache, pool.tables[0], [0], [0, 1], pool.tables[1], [2, 2], *pool.scale,
                                    pool.softmax_scale, m, s)
        out, lse = _call(pool, q, [0], [0, 1], [2, 2], m, s)
        assert bool((out == 0).all())
        assert inputs.within(out, lse, want, 2) is None


@pytest.mark.parametrize("page", [16, 64, 256])
def test_a_long_prefix_in_many_pieces(page):
    _check(4, [6001], [0, 3], [20, 300, 7], 1, 4, 128, page, False)
    _check(5, [3000, 2500], [0, 1, 4], [1, 5, 70, 600], 1, 5, 64, page, True, q_len=2)


@pytest.mark.parametrize("count", [33, 700])
def test_many_sequences_and_prefixes(count):
    rng = np.random.default_rng(count)
    cuts = np.sort(rng.choice(count + 1, min(count, 40), replace=False))
    _check(6, rng.integers(0, 60, len(cuts) - 1).tolist(), cuts.tolist(), rng.integers(0, 30, count).tolist(), 1, 1, 64,
           16, False)


def test_a_nan_reaches_the_rows_that_see_it():
    lens = [20, 25, 9]
    pool, q, _, _, _ = inputs.shared_case(7, [90], [0, 2], lens, 1, 2, 64, 16, False, 3)
    clean = inputs.ragged.shared(q, *pool.cache, pool.tables[0], [90], [0, 2], pool.tables[1], lens, *pool.scale,
                                 pool.softmax_scale)
    # the second sequence's last key is hidden from its first two tokens: a NaN in its K and in its V
    pool.cache[0][pool.tables[1][1, 1], 0, 8, 5] = 0x7F
    pool.cache[1][pool.tables[1][1, 1], 0, 8, 6] = 0x7F
    out, lse = _call(pool, q, [90], [0, 2], lens)
    assert bool(out[1, 2].isnan().all()) and bool(lse[1, 2].isnan().all()) and int(lse.isnan().sum()) == 2
    out[1, 2], lse[1, 2] = torch.from_numpy(clean[0][5]).to(DEV), torch.from_numpy(clean[1][5]).to(DEV)
    assert inputs.within(out, lse, clean, 115) is None
    pool.cache[0][pool.tables[1][1, 1], 0, 8, 5] = 0x10
    out, lse = _call(pool, q, [90], [0, 2], lens)
    assert int(out.isnan().sum()) == 2 and bool(out[1, 2, :, 6].isnan().all())  # V alone: that dim
    pool.cache[1][pool.tables[0][0, 1], 0, 0, 0] = 0x7F
    out, lse = _call(pool, q, [90], [0, 2], lens)
    assert bool(out[:2, :, :, 0].isnan().all()) and not bool(out[2].isnan().any())


def test_errors_in_place_and_replay():
    lens = [50, 3, 130, 0]
    pool, q, m, s, want = inputs.shared_case(8, [170, 40], [0, 2, 3], lens, 2, 3, 128, 32, True, 2, True, True)
    first = _call(pool, q, [170, 40], [0, 2, 3], lens, m, s)
    assert inputs.within(*first, want, 300) is None
    here = q.to(DEV)
    got, _ = _call(pool, here, [170, 40], [0, 2, 3], lens, m, s, out=here)
    assert got is here and torch.equal(here, first[0])
    out, lse = _call(pool, q, [170, -2], [0, 2, 3], lens, m, s)
    assert fm.last_device_error() == fm.DEV_BAD_SEQLEN
    keep = np.r_[0:4, 6:8]  # the second prefix counts as empty
    flat = lambda x: x.reshape(8, *x.shape[2:])[keep]  # noqa: E731
    assert inputs.within(flat(out), flat(lse), [w[keep] for w in want], 300) is None
    k, v, ptable, table, ks, vs = pool.device(DEV)
    ins = (q.to(DEV), k, v, ptable, _i32([170, 40]), _i32([0, 2, 3]), table, _i32(lens), ks, vs)
    kw = dict(softmax_scale=pool.softmax_scale, spec_mask=torch.from_numpy(m).to(DEV), sinks=torch.from_numpy(s).to(DEV))
    ws = torch.empty(fm.gqa_shared_workspace_bytes(4, 2, 6, 2, 128, 2, ptable.shape[1] * 32, table.shape[1] * 32),
                     dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fm.paged_gqa_decode_shared(*ins, **kw, out=out, lse=lse, workspace=ws)
    for _ in range(2):
        out.zero_(), ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    pool.tables[0][0, 2] = -5
    _call(pool, q, [170, 40], [0, 2, 3], lens, m, s)
    assert fm.last_device_error() == fm.DEV_BAD_PAGE


def test_a_step_with_the_other_calls():
    """A decode step of four samples of one prompt: rows appended, then attended behind the shared prompt; the same from
    cross attention to the prompt, a decode over the own keys and the merge; and from a decode that holds the prompt for
    each sample."""
    g = torch.Generator().manual_seed(1)
    hd, page, h_kv, h_q, prompt, own = 128, 16, 2, 8, 96, [5, 17, 1, 40]
    blocks = prompt // page + sum(-(-n // page) for n in own)
    rows = lambda n, h: torch.randn((n, h, hd), generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    caches = [torch.zeros((blocks, h_kv, page, hd), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    unit = torch.tensor([0.02], device=DEV)
    f, factor = fm.rotary_frequencies(hd)
    table = fm.rotary_table(f, 256, factor=factor)
    perm = torch.randperm(blocks, generator=g)
    ptable = perm[:prompt // page].reshape(1, -1)
    otable, at = torch.zeros((4, 3), dtype=torch.int64), prompt // page
    for b, n in enumerate(own):
        c = -(-n // page)
        otable[b, :c] = perm[at:at + c]
        at += c

    def append(t, first, count, q=None):
        j = torch.arange(first, first + count)
        slots = (t[j // page] * page + j % page).to(torch.int32).to(DEV)
        base = 0 if t is ptable[0] else prompt
        return fm.paged_kv_append(rows(count, h_kv), rows(count, h_kv), slots, *caches, positions=(j + base).to(DEV),
                                  table=table, k_scale=unit, v_scale=unit, q=q)

    append(ptable[0], 0, prompt)
    q = torch.cat([append(otable[b], 0, n, rows(n, h_q))[-1:] for b, n in enumerate(own)])
    lens = _i32(own)
    out, lse = fm.paged_gqa_decode_shared(q, *caches, _i32(ptable), _i32([prompt]), _i32([0, 4]), _i32(otable), lens, unit,
                                          unit)
    front = fm.paged_cross_attention(q, *caches, _i32(ptable), _i32([prompt]), unit, unit, q_starts=_i32([0, 4]))
    back = fm.paged_gqa_decode(q, *caches, _i32(otable), lens, unit, unit)
    joined = fm.attention_merge([front[0], back[0]], [front[1], back[1]])
    both = torch.cat((ptable.expand(4, -1), otable), 1)
    whole = fm.paged_gqa_decode(q, *caches, _i32(both), lens + prompt, unit, unit)
    torch.cuda.synchronize()
    assert fm.last_device_error() == 0
    want = inputs.ragged.shared(q.cpu().unsqueeze(1), caches[0].cpu(), caches[1].cpu(), ptable.numpy(), [prompt], [0, 4],
                                otable.numpy(), own, 0.02, 0.02, hd ** -0.5)
    assert inputs.within(out, lse, want, 140) is None
    # the older decode keeps Q and P to 8 bits each (2^-8 of a weight), the merge takes parts rounded to bf16 (2^-8 each)
    for o, l in (joined, whole):
        assert np.all(np.abs(o.double().cpu().numpy() - want[0]) <= 2.0 ** -7 * np.abs(want[0]) + 2.0 ** -6 * want[2])
        assert np.all(np.abs(l.double().cpu().numpy() - want[1]) <= 1e-3)


@pytest.mark.parametrize("hd,h_q,bs", [(64, 3, 1), (64, 3, 3), (128, 3, 1), (128, 1, 3)])
def test_blocks_in_place_of_odd_numbers_of_rows(hd, h_q, bs):
    """Blocks whose result takes the queries' place, with rows that are no multiple of what a thread block joins."""
    lens = [40, 3, 130][:bs]
    pool, q, m, s, want = inputs.shared_case(9, [70], [0, bs], lens, 1, h_q, hd, 16, False, 3, True)
    first = _call(pool, q, [70], [0, bs], lens, m, s)
    assert inputs.within(*first, want, 200) is None
    for _ in range(20):
        here = q.to(DEV)
        out, lse = _call(pool, here, [70], [0, bs], lens, m, s, out=here)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("hd,rows", [(64, False), (128, True)])
@pytest.mark.parametrize("q_len", [1, 9])
def test_more_rows_than_are_joined_at_a_time(hd, rows, q_len):
    """Past the rows from which a row is joined by half as many lanes (4864 of 128 dims, 9728 of 64)."""
    bs = 1300 if q_len == 1 else 190
    lens = np.random.default_rng(11).integers(0, 40, bs).tolist()
    _check(11, [150, 9], [0, bs // 2, bs - 20], lens, 2, 4, hd, 16, rows, q_len=q_len, mask=q_len > 1, sinks=True)


@pytest.mark.parametrize("hd,q_len", [(64, 1), (128, 3)])
def test_no_prefixes(hd, q_len):
    """A batch in which nothing is shared: tables of no rows."""
    _check(14, [], [0], [3, 40, 0, 200], 2, 2, hd, 16, False, q_len=q_len, sinks=True)
