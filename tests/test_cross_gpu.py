"""Cross attention on the GPU against the float64 oracle (tolerances: tests/ragged_inputs.py)."""

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from tests import ragged_inputs as inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _call(pool, q, kv_lens, starts, **kw):
    k, v, table, ks, vs = pool.device(DEV)
    out, lse = fm.paged_cross_attention(
        q.to(DEV) if not q.is_cuda else q, k, v, table, torch.tensor(kv_lens, dtype=torch.int32, device=DEV), ks, vs,
        softmax_scale=pool.softmax_scale,
        q_starts=None if starts is None else torch.from_numpy(np.asarray(starts, np.int32)).to(DEV), **kw)
    torch.cuda.synchronize()
    return out, lse


def _check(seed, q_lens, kv_lens, h_kv, group, hd, page, rows, pad=(0, 0), size=1.0):
    pool, q, starts, want = inputs.cross_case(seed, q_lens, kv_lens, h_kv, group, hd, page, rows, pad, size)
    out, lse = _call(pool, q, kv_lens, starts)
    wrong = inputs.within(out, lse, want, max([1, *kv_lens]))
    assert wrong is None, wrong
    assert fm.last_device_error() == 0


# rows of an item: one, a quarter of the lanes and past it, one stream and past it, two streams and past them; keys: one,
# a tile and past it, several; one head, odd groups, wide ones
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("q_lens,kv_lens,h_kv,group", [
    ([1], [1], 1, 1), ([1], [128], 2, 4), ([2], [129], 1, 8), ([32], [127], 1, 1), ([33], [300], 1, 1),
    ([128], [256], 1, 1), ([43], [257], 1, 3), ([255], [65], 1, 1), ([256], [384], 1, 1), ([37], [400], 1, 7),
    ([300], [130], 2, 1), ([5, 0, 1, 70, 130, 3], [17, 40, 0, 129, 260, 128], 2, 2)])
def test_shapes(q_lens, kv_lens, h_kv, group, hd, rows):
    _check(1, q_lens, kv_lens, h_kv, group, hd, 16, rows)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hd,rows", [(64, True), (128, False)])
def test_pages(page, hd, rows):
    """Lengths that end inside a page, on its last key and on a page's border inside a tile."""
    _check(page, [4, 40, 1, 9], [1, page, page + 1, 3 * page - 1], 2, 2, hd, page, rows)


@pytest.mark.parametrize("hd,rows,group,tokens", [(128, False, 4, 1), (128, True, 16, 5), (64, False, 1, 1), (64, True, 3, 50)])
def test_few_long_items_are_cut(hd, rows, group, tokens):
    """Fewer items than CTAs: every one lies in several shares."""
    _check(7, [tokens, tokens], [5000, 3111], 1, group, hd, 64, rows)


@pytest.mark.parametrize("count", [31, 33, 600, 2100])
def test_many_sequences(count):
    """More sequences than lanes, than threads, than groups of 32 whose places are kept; some without keys or tokens."""
    rng = np.random.default_rng(count)
    _check(8, rng.integers(0, 3, count).tolist(), rng.integers(0, 40, count).tolist(), 1, 1, 64, 16, False)


@pytest.mark.parametrize("seed", range(6))
def test_mixed_batches(seed):
    """Items of all forms next to each other, with and without keys, whole and cut."""
    rng = np.random.default_rng(100 + seed)
    n = int(rng.integers(2, 30))
    q_lens = np.where(rng.random(n) < 0.5, rng.integers(0, 12, n), rng.integers(30, 150, n))
    kv_lens = np.where(rng.random(n) < 0.3, 0, rng.integers(1, 500, n))
    _check(seed, q_lens.tolist(), kv_lens.tolist(), int(rng.integers(1, 4)), int(rng.integers(1, 4)),
           int(rng.choice([64, 128])), int(rng.choice([16, 64])), bool(seed % 2))


def test_one_token_each():
    pool, q, starts, want = inputs.cross_case(9, [1] * 5, [0, 1, 200, 77, 128], 2, 4, 128, 32, True)
    out, lse = _call(pool, q, [0, 1, 200, 77, 128], None)
    assert inputs.within(out, lse, want, 200) is None


def test_tokens_of_no_sequence():
    """Zeros and -inf in outputs that the call makes; given ones keep their rows."""
    lens = [30, 0, 50]
    pool, q, starts, want = inputs.cross_case(10, [3, 2, 4], lens, 1, 2, 64, 16, False, pad=(2, 5))
    out, lse = _call(pool, q, lens, starts)
    assert inputs.within(out, lse, want, 50) is None
    out = torch.full_like(q.to(DEV), 7.0)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    _call(pool, q, lens, starts, out=out, lse=lse)
    for a in (slice(0, 2), slice(11, 16)):
        assert bool((out[a] == 7).all()) and bool((lse[a] == 5).all())
        out[a], lse[a] = 0, -float("inf")
    assert inputs.within(out, lse, want, 50) is None


@pytest.mark.parametrize("strides", [(3 * 2 * 64, 64), (64, 12 * 64), (200, 72)])
def test_strided_queries_and_outputs(strides):
    """Heads of one projection's rows, tokens of each head together, and gaps; the output in the queries' place."""
    lens = [100, 60]
    pool, q, starts, want = inputs.cross_case(11, [7, 5], lens, 1, 2, 64, 16, False)
    buf = torch.full((16 * 1024,), 3.0, dtype=torch.bfloat16, device=DEV)
    at = buf[64:].as_strided((12, 2, 64), (*strides, 1))
    at.copy_(q)
    before = buf.clone()
    out, lse = _call(pool, at, lens, starts)
    assert inputs.within(out, lse, want, 100) is None and torch.equal(buf, before)
    got, _ = _call(pool, at, lens, starts, out=at)
    assert got is at and torch.equal(at, out)
    at.copy_(q)
    assert torch.equal(buf, before)  # nothing between the rows was written


def test_a_nan_stays_in_its_sequence():
    lens = [150, 150, 40]
    pool, q, starts, want = inputs.cross_case(12, [40, 3, 2], lens, 1, 1, 128, 16, False)
    pool.cache[0][pool.tables[0][1, 2], 0, 5, 9] = 0x7F   # a key of the second sequence
    pool.cache[1][pool.tables[0][2, 1], 0, 3, 17] = 0xFF  # a value of the third
    out, lse = _call(pool, q, lens, starts)
    assert bool(out[40:43].isnan().all()) and bool(lse[40:43].isnan().all())
    assert bool(out[43:, 0, 17].isnan().all()) and int(out[43:].isnan().sum()) == 2
    assert bool(torch.isfinite(lse[43:]).all())
    part = [w[:40] for w in want]
    assert inputs.within(out[:40], lse[:40], part, 150) is None


def test_a_nan_query_stays_in_its_row():
    lens = [150]
    pool, q, starts, want = inputs.cross_case(13, [140], lens, 1, 2, 64, 16, True)
    q[17, 1, 3], q[100, 0, 0] = float("nan"), float("inf")
    out, lse = _call(pool, q, lens, starts)
    for t, h in ((17, 1), (100, 0)):
        assert bool(out[t, h].isnan().all()) and bool(lse[t, h].isnan())
        out[t, h], lse[t, h] = torch.from_numpy(want[0][t, h]).to(DEV), float(want[1][t, h])
    assert inputs.within(out, lse, want, 150) is None


@pytest.mark.parametrize("power", [-70, -30, 12, 24, 40, 60])
@pytest.mark.parametrize("tokens", [1, 40, 140])
def test_queries_of_any_size(power, tokens):
    """Far scores: where the best key leads by much, its value comes back; tiny ones: the mean of the values."""
    pool, q, starts, want = inputs.cross_case(14, [tokens], [300], 1, 1, 64, 16, False, size=2.0 ** power)
    out, lse = _call(pool, q, [300], starts)
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got)) and bool(torch.isfinite(lse).all())
    if power < 0:
        assert inputs.within(out, lse, want, 300) is None
        return
    k = inputs.ragged.gather(pool.cache[0], pool.scale[0], pool.tables[0][0], 300, 0)
    v = inputs.ragged.gather(pool.cache[1], pool.scale[1], pool.tables[0][0], 300, 0)
    s = q[:, 0].double().numpy() @ k.T * pool.softmax_scale
    order = np.sort(s, 1)
    # the score's error is 2^-16 of its terms (tests/ragged_inputs.py); 20 units of lead leave 300 e^-20 to the others
    size = (np.abs(q[:, 0].double().numpy()) + np.abs(q[:, 0].double().numpy()).max(1, keepdims=True) / 4) @ np.abs(k).T
    lead = order[:, -1] - order[:, -2] > 20 + 2.0 ** -14 * size.max(1) * pool.softmax_scale
    assert lead.any() or power < 24
    best = v[s.argmax(1)]
    assert np.all(np.abs(got[lead, 0] - best[lead]) <= 2.0 ** -8 * np.abs(best[lead]) + 1e-5)


def test_equal_scores_and_equal_keys():
    """A query of zeros weighs all keys alike."""
    pool, q, starts, _ = inputs.cross_case(15, [60], [333], 1, 1, 128, 16, True)
    q.zero_()
    want = inputs.ragged.cross(q, *pool.cache, pool.tables[0], [333], *pool.scale, pool.softmax_scale, starts)
    out, lse = _call(pool, q, [333], starts)
    assert inputs.within(out, lse, want, 333) is None


def test_growing_scores():
    """Keys whose scores rise by tens from tile to tile: the reference moves again and again, in every form."""
    for tokens in (2, 60, 200):
        pool, q, starts, _ = inputs.cross_case(16, [tokens], [900], 1, 1, 64, 16, False)
        grow = inputs.e4m3_encode(np.linspace(0.0, 400.0, 900))
        q[..., 0] = 100.0
        pool.cache[0][:] &= 0x07  # small keys, but for the first dim
        for j in range(900):
            pool.cache[0][pool.tables[0][0, j // 16], 0, j % 16, 0] = grow[j]
        want = inputs.ragged.cross(q, *pool.cache, pool.tables[0], [900], *pool.scale, pool.softmax_scale, starts)
        out, lse = _call(pool, q, [900], starts)
        wrong = inputs.within(out, lse, want, 900)
        assert wrong is None, (tokens, wrong)


def test_bad_lengths_starts_and_pages():
    """What does not fit counts as empty, or reads page 0, and says so."""
    lens = [40, 33, 20]
    pool, q, starts, want = inputs.cross_case(17, [4, 4, 4], lens, 1, 2, 64, 16, False)
    for bad_lens in ([40, -1, 20], [40, 1000, 20]):
        out, lse = _call(pool, q, bad_lens, starts)
        assert fm.last_device_error() == fm.DEV_BAD_SEQLEN
        assert bool((out[4:8] == 0).all()) and bool((lse[4:8] == -float("inf")).all())
        keep = np.r_[0:4, 8:12]
        assert inputs.within(out[keep], lse[keep], [w[keep] for w in want], 40) is None
    out, lse = _call(pool, q, lens, [0, 4, 8, 13])  # the last range passes the tokens
    assert fm.last_device_error() == fm.DEV_BAD_SEQLEN
    assert inputs.within(out[:8], lse[:8], [w[:8] for w in want], 40) is None
    pool.tables[0][1, 1] = pool.cache[0].shape[0]
    _call(pool, q, lens, starts)
    assert fm.last_device_error() == fm.DEV_BAD_PAGE


def test_replayed_and_on_two_streams():
    """The same bits from a captured graph, from two streams at once, and again."""
    lens = [700, 0, 300, 129]
    pool, q, starts, want = inputs.cross_case(18, [140, 3, 20, 33], lens, 2, 2, 128, 16, True)
    k, v, table, ks, vs = pool.device(DEV)
    args = (q.to(DEV), k, v, table, torch.tensor(lens, dtype=torch.int32, device=DEV), ks, vs)
    kw = dict(softmax_scale=pool.softmax_scale, q_starts=torch.from_numpy(starts).to(DEV))
    first = fm.paged_cross_attention(*args, **kw)
    torch.cuda.synchronize()
    assert inputs.within(*first, want, 700) is None
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for s in streams:
        with torch.cuda.stream(s):
            results.append([fm.paged_cross_attention(*args, **kw) for _ in range(5)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, first[0]) and torch.equal(l, first[1]) for r in results for o, l in r)
    graph = torch.cuda.CUDAGraph()
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    ws = torch.empty(fm.cross_workspace_bytes(q.shape[0], 4, 4, 2, 128, table.shape[1] * 16), dtype=torch.uint8, device=DEV)
    with torch.cuda.graph(graph):
        fm.paged_cross_attention(*args, **kw, out=out, lse=lse, workspace=ws)
    for _ in range(3):
        out.zero_(), lse.zero_(), ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    args[4].fill_(100)  # the lengths are read when the graph runs
    graph.replay()
    want = inputs.ragged.cross(q, *pool.cache, pool.tables[0], [100] * 4, *pool.scale, pool.softmax_scale, starts)
    torch.cuda.synchronize()
    assert not torch.equal(out, first[0]) or lens == [100] * 4
    assert inputs.within(out[:140], lse[:140], [w[:140] for w in want], 100) is None


def test_no_tokens_and_no_sequences():
    pool, q, starts, _ = inputs.cross_case(19, [3], [20], 1, 2, 64, 16, False)
    out, lse = _call(pool, q[:0], [20], [0, 0])
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    k, v, table, ks, vs = pool.device(DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    out, lse = fm.paged_cross_attention(q.to(DEV), k, v, table[:0], none, ks, vs,
                                        q_starts=torch.zeros(1, dtype=torch.int32, device=DEV))
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    assert fm.last_device_error() == 0


def test_a_line_past_32_bits():
    """One head's items add up to more than 2^31 of the units in which work is shared: 11250 of 8192 tiles.

    512 times the same 2048 keys leave the output as it is and lift lse by log 512.  Either output is off by half a step
    of bf16, 2^-8 of it, and 2^-11 of the largest value for P in f16; the long sum also by its 65536 additions of 16 keys
    in 32 bits (2^-23 each of the sum of |p v|, if they truncate), its l by 8192 of them (2^-24).
    """
    tokens, h_q, hd, page = 45000, 64, 64, 256
    gen = torch.Generator(device=DEV).manual_seed(5)
    k, v = (torch.randn(8, 1, page, hd, generator=gen, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    q = (3 * torch.randn(tokens, h_q, hd, generator=gen, device=DEV)).to(torch.bfloat16)
    table = (torch.arange(4096, device=DEV, dtype=torch.int32) % 8)[None].contiguous()
    one, starts = torch.ones(1, device=DEV), torch.tensor([0, tokens], dtype=torch.int32, device=DEV)
    short, long = (fm.paged_cross_attention(q, k, v, table, torch.tensor([n], dtype=torch.int32, device=DEV), one, one,
                                            softmax_scale=hd ** -0.5, q_starts=starts) for n in (2048, 1 << 20))
    want, got = short[0].float(), long[0].float()
    largest = float(v.float().abs().max())
    assert bool(((got - want).abs() <= want.abs() * 2 ** -7 + largest * (2 ** -10 + 2 ** -7)).all())
    assert float((long[1] - short[1] - np.log(512)).abs().max()) <= 2 ** -10
    assert fm.last_device_error() == 0


@pytest.mark.parametrize("tokens,bs,h_kv,group,hd,rows,keys", [
    (1, 1, 16, 1, 64, False, 1024), (1, 1, 16, 1, 64, False, 1153), (1, 19, 8, 4, 128, True, 600),
    (1, 20, 8, 4, 128, True, 600), (200, 2, 4, 1, 64, False, 384), (200, 2, 4, 1, 64, False, 400)])
def test_around_the_border_of_whole_items(tokens, bs, h_kv, group, hd, rows, keys):
    """Calls of few short items, which are not cut and merged, and calls just past them."""
    rng = np.random.default_rng(keys)
    lens = rng.integers(0, keys + 1, bs)
    lens[0] = keys
    _check(12, [tokens] * bs, lens.tolist(), h_kv, group, hd, 16, rows)
    pool, q, _, want = inputs.cross_case(13, [1] * bs, lens.tolist(), h_kv, group, hd, 16, rows)
    assert inputs.within(*_call(pool, q, lens.tolist(), None), want, keys) is None
