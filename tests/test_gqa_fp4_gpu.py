"""Paged GQA decode over the 4-bit cache on the GPU against the float64 oracle.

Tolerances, before any run.  Scores: K and Q enter exactly; a product of
head_dim terms is summed in float32, at most head_dim + 2 roundings of 2^-23
(tensor-core sums may truncate) of S = scale sum |q| |k|, so a score is off by
e = (head_dim + 4) 2^-23 max S and the LSE by no more than that, plus the
approximate 2^x and log2 (2^-21 together) and its own rounding.  Outputs: a
weight is off by the f16 rounding 2^-11, by 2 e (its own score and the sum's)
and 2^-20 of approximate functions and float32 sums, against sum p |v|; then
the rounding to bf16, 2^-8 of the value.  f16's normal numbers end at 2^-14 and
its spacing below is 2^-24: the largest weight is stored as 2^7 or more, so a
small weight is off by at most 2^-25 / 2^7 = 2^-32 of the largest, which adds
keys * 2^-32 * max |v|.
"""

import math

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from oracle import fp4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


class Inputs:
    """Seeded caches of unequal contexts: used blocks at a random permutation of the pool; spare blocks
    and slots past a sequence's end hold NaN scales and every code."""

    def __init__(self, seed, lens, h_kv, group, hd, page, q_len=1, mask=False, sinks=False, spare=3):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        bs = len(lens)
        n_blocks = (self.lens + page - 1) // page
        used = int(n_blocks.sum())
        total = used + spare
        perm = rng.permutation(total)
        self.bt = np.full((bs, max(1, int(n_blocks.max()))), perm[-1], np.int32)
        valid = np.zeros((total, page), bool)
        at = 0
        for b in range(bs):
            for p in range(n_blocks[b]):
                self.bt[b, p] = perm[at]
                valid[perm[at], :min(page, self.lens[b] - p * page)] = True
                at += 1
        self.codes, self.s8, self.scale = [], [], []
        for _ in range(2):
            x = rng.standard_normal((total, h_kv, page, hd)).astype(np.float32)
            x *= np.exp(0.5 * rng.standard_normal(hd)).astype(np.float32)  # some dims larger than others
            scale = float(np.float32(np.abs(x).max() / (448 * 6)))
            codes, s8 = fp4.quantise(x, scale)
            bad = ~np.broadcast_to(valid[:, None], (total, h_kv, page))
            codes[bad] = rng.integers(0, 256, (int(bad.sum()), hd // 2)).astype(np.uint8)
            s8[bad] = np.where(rng.random((int(bad.sum()), hd // 16)) < 0.5, 0x7F, 0xFF)
            self.codes.append(codes), self.s8.append(s8), self.scale.append(scale)
        self.q = torch.from_numpy(rng.standard_normal((bs, q_len, h_kv * group, hd))).to(torch.bfloat16)
        self.mask = None
        if mask:
            m = rng.random((bs, q_len, q_len)) < 0.5
            self.mask = torch.from_numpy(m.astype(np.uint8))
        self.sinks = torch.from_numpy(rng.standard_normal(h_kv * group).astype(np.float32)) if sinks else None
        self.softmax_scale = float(np.float32(1 / math.sqrt(hd)))
        self.hd = hd

    def run(self, **kw):
        d = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
        args = [self.q.to(DEV), d(self.codes[0]), d(self.codes[1]), d(self.s8[0]).view(torch.float8_e4m3fn),
                d(self.s8[1]).view(torch.float8_e4m3fn), d(self.bt), d(self.lens),
                torch.tensor([self.scale[0]], device=DEV), torch.tensor([self.scale[1]], device=DEV)]
        out, lse = fm.paged_gqa_decode_fp4(*args, softmax_scale=self.softmax_scale,
                                           spec_mask=None if self.mask is None else self.mask.to(DEV),
                                           sinks=None if self.sinks is None else self.sinks.to(DEV), **kw)
        torch.cuda.synchronize()
        return out, lse

    def want(self, window=0, rows=None):
        return fp4.gqa_decode(self.q, self.codes[0], self.codes[1], self.s8[0], self.s8[1], self.bt, self.lens,
                              self.scale[0], self.scale[1], self.softmax_scale, self.mask, window, self.sinks, rows)

    def check(self, out, lse, window=0, rows=None):
        o, l, a = self.want(window, rows)
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        used = np.zeros(self.codes[0].shape[0], bool)
        for b, n in enumerate(self.lens):
            used[self.bt[b, :-(-int(n) // self.codes[0].shape[2])]] = True
        sizes = [np.abs(fp4.dequantise(self.codes[i][used], np.where(self.s8[i][used] & 0x7F == 0x7F, 0,
                                                                    self.s8[i][used]), self.scale[i])) for i in (0, 1)]
        kmax = np.sqrt((sizes[0] ** 2).sum(-1)).max() if used.any() else 0.0
        vmax = sizes[1].max() if used.any() else 0.0
        qmax = float(self.q.double().norm(dim=-1).max())
        e = (self.hd + 4) * 2.0 ** -23 * self.softmax_scale * kmax * qmax  # |q| |k| bounds sum |q_d k_d|
        pick = slice(None) if rows is None else tuple(np.array(rows).T)
        sel = lambda x: x if rows is None else np.moveaxis(x, 2, 1)[pick]  # noqa: E731
        o, l, a, got, gl = sel(o), sel(l), sel(a), sel(got), sel(gl)
        empty = np.isneginf(l)
        assert np.all(np.isneginf(gl[empty])) and np.all(got[empty] == 0)
        assert np.all(np.isfinite(gl[~empty])) and np.all(np.isfinite(got))
        dl, al = np.abs(gl[~empty] - l[~empty]), np.abs(l[~empty])
        assert np.all(dl <= e + 2.0 ** -21 + 2.0 ** -23 * al), (dl.max(), e)
        tol = 2.0 ** -8 * np.abs(o) + (1 + 2.0 ** -8) * (a * (2.0 ** -11 + 2 * e + 2.0 ** -20) +
                                                         int(self.lens.max()) * 2.0 ** -32 * vmax)
        assert np.all(np.abs(got - o) <= tol), float(np.max(np.abs(got - o) / tol))
        assert fm.last_device_error() == 0


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 7, 8, 16])
def test_ragged(hd, group):
    x = Inputs(hd + group, [300, 0, 1, 16, 17, 2000, 129], 2, group, hd, 16)
    for splits in (0, 1, 5):
        x.check(*x.run(num_splits=splits))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages(page):
    x = Inputs(page, [1, 700, 15, page, page + 1, 0], 3, 3, 64, page)
    x.check(*x.run())
    x = Inputs(page + 1, [1100, 33], 1, 4, 128, page)
    x.check(*x.run(num_splits=3))


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [31], [128], [129], [0]])
def test_single_sequences(lens):
    x = Inputs(5, lens, 8, 4, 128, 16)
    x.check(*x.run())


def test_a_small_grid_is_split_and_merged():
    """One sequence of one KV head: the keys are cut over the GPU; every forced count agrees too."""
    x = Inputs(6, [9001], 1, 4, 128, 16)
    assert fm.gqa_fp4_workspace_bytes(1, 4, 1, 128, 9008) > 0
    for splits in (0, 1, 2, 3, 16, 60, 1000):
        x.check(*x.run(num_splits=splits))


OPTIONS = [  # q_len, group, mask, window, sinks, hd, splits
    (1, 4, False, 0, True, 128, 0),
    (1, 8, False, 37, False, 128, 1),
    (1, 1, False, 1, False, 64, 2),
    (2, 4, False, 0, False, 128, 3),
    (4, 4, True, 0, False, 128, 1),
    (4, 4, True, 100, True, 128, 2),
    (3, 5, False, 300, True, 64, 1),
    (3, 5, True, 2, False, 256, 1),
    (16, 1, True, 0, True, 64, 4),
    (16, 8, True, 50, True, 128, 1),     # 128 columns: eight column tiles
    (5, 12, False, 0, False, 64, 2),     # 60 columns: the last tile is partly empty
    (1, 64, False, 0, False, 128, 0),
    (1, 2, True, 0, False, 128, 1),      # a token that its own mask may hide
]


@pytest.mark.parametrize("q_len,group,mask,window,sinks,hd,splits", OPTIONS)
def test_blocks_windows_and_sinks(q_len, group, mask, window, sinks, hd, splits):
    # caches shorter than the block, empty, on and off a tile's end
    x = Inputs(q_len * 100 + group + window, [700, 3, 0, 48, 1, 129], 2, group, hd, 16, q_len, mask, sinks)
    x.check(*x.run(window=window, num_splits=splits), window=window)


def test_a_window_longer_than_every_sequence_hides_nothing():
    x = Inputs(60, [700, 48, 0, 3, 3000], 2, 4, 64, 16, 3)
    for splits in (0, 1, 3):
        want, want_lse = x.run(num_splits=splits)
        for window in (3008, 1 << 30, (1 << 31) - 1):
            out, lse = x.run(num_splits=splits, window=window)
            assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_rows_that_see_nothing():
    """A block whose mask hides everything from a token of a cache no longer than the block: zeros and -inf,
    or the sink's logit."""
    for sinks in (False, True):
        x = Inputs(9, [4, 2], 1, 2, 64, 16, q_len=4, mask=True, sinks=sinks)
        x.mask[0, 1] = 0
        x.mask[1] = 0
        out, lse = x.run()
        x.check(out, lse)
        assert torch.all(out[0, 1] == 0) and torch.all(out[1] == 0)
        want = x.sinks if sinks else torch.full((2,), -math.inf)
        assert torch.allclose(lse[0, 1].cpu(), want)


def test_hidden_keys_may_hold_anything():
    """NaN scales on keys that no token sees -- hidden by the mask, or left behind by the window -- change nothing;
    with 60 columns each column tile has its own set of tokens."""
    for q_len, group, window in ((4, 4, 0), (4, 4, 3), (5, 12, 0), (5, 12, 40), (1, 4, 0)):
        x = Inputs(20 + group + window, [700, 40, 5, 2000], 2, group, 128, 16, q_len, mask=True)
        x.mask[:, :, q_len - 1] = 0  # the block's last key is hidden from every token ...
        if q_len == 5:
            x.mask[:, :, 1] = 0
            x.mask[:, 4, 1] = 1      # ... and the second from all but the last, of another column tile than the first
        for b, n in enumerate(x.lens):
            hidden = [n - 1] + ([n - q_len - window] if window and n > window + q_len else [])
            for j in hidden:
                for s8 in x.s8:
                    s8[x.bt[b, j // 16], :, j % 16] = 0x7F
        for splits in (0, 1, 2):
            x.check(*x.run(window=window, num_splits=splits), window=window)


@pytest.mark.parametrize("q_len,group,mask,window,sinks", [(1, 4, False, 0, True), (4, 4, True, 1500, True),
                                                           (4, 4, True, 1600, True), (3, 7, False, 100, False),
                                                           (16, 8, True, 0, True)])
def test_balanced_pieces_with_options(q_len, group, mask, window, sinks):
    """Contexts long and unequal enough that the keys are cut on the device, at cuts of its own choosing."""
    x = Inputs(30 + q_len + window, [5000, 0, 3, 1700, 2900, 17], 2, group, 64, 16, q_len, mask, sinks)
    # (these windows leave so little that clusters take the sequences uncut)
    assert (fm.gqa_fp4_workspace_bytes(6, 2 * group, 2, 64, x.bt.shape[1] * 16, q_len, window) > 0) == (window == 0)
    x.check(*x.run(window=window), window=window)


@pytest.mark.parametrize("q_len,group,mask,window,sinks", [(4, 4, True, 8100, True), (3, 7, False, 5000, False)])
def test_balanced_pieces_with_windows(q_len, group, mask, window, sinks):
    x = Inputs(35 + q_len, [9000, 0, 3, 4700, 2900, 17], 2, group, 64, 16, q_len, mask, sinks)
    assert fm.gqa_fp4_workspace_bytes(6, 2 * group, 2, 64, x.bt.shape[1] * 16, q_len, window) > 0
    x.check(*x.run(window=window), window=window)


# Sequences in clusters of eight, four and two CTAs: (sequences, KV heads) give the size.
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("bs,h_kv", [(5, 2), (7, 4), (14, 5)])
@pytest.mark.parametrize("q_len,group,mask,window,sinks", [(1, 5, False, 0, True), (1, 16, False, 900, False),
                                                           (4, 3, True, 0, False), (5, 2, True, 700, True)])
def test_clusters(hd, bs, h_kv, q_len, group, mask, window, sinks):
    """Contexts of none, of fewer tiles than a cluster has warps, on and off its last tile, and of several rounds."""
    lens = ([1600, 0, 1, 17, 1025] + [33 * i for i in range(20)])[:bs]
    x = Inputs(200 + hd + bs + q_len + group, lens, h_kv, group, hd, 16, q_len, mask, sinks)
    assert fm.gqa_fp4_workspace_bytes(bs, h_kv * group, h_kv, hd, x.bt.shape[1] * 16, q_len, window) == 0
    rows = [(b, h) for b in range(5) for h in (0, h_kv * group - 1)] + [(bs - 1, group)]
    out, lse = x.run(window=window)
    x.check(out, lse, window=window, rows=rows)
    one, lse1 = x.run(window=window, num_splits=1)  # the same sums in another order
    live = torch.isfinite(lse1)
    assert torch.equal(live, torch.isfinite(lse))
    assert torch.all((lse[live] - lse1[live]).abs() <= 2.0 ** -16)
    assert torch.all((out - one).abs().float() <= 2.0 ** -7 * one.abs().float() + 2.0 ** -9)
    again, lse2 = x.run(window=window)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("bs", [6, 16, 30])
def test_clusters_of_sixteen_columns(hd, bs):
    """Contexts too long for tiles of eight columns and too short to be cut: clusters of eight, four and two CTAs."""
    x = Inputs(300 + hd + bs, ([2500, 0, 15, 2065] + [33 * i for i in range(30)])[:bs], 2, 4, hd, 16, 4, mask=True)
    assert fm.gqa_fp4_workspace_bytes(bs, 8, 2, hd, x.bt.shape[1] * 16, 4) == 0
    out, lse = x.run()
    x.check(out, lse, rows=[(b, h) for b in range(4) for h in (0, 5)] + [(bs - 1, 7)])
    one, lse1 = x.run(num_splits=1)  # the same sums in another order
    live = torch.isfinite(lse1)
    assert torch.equal(live, torch.isfinite(lse)) and torch.all((lse[live] - lse1[live]).abs() <= 2.0 ** -16)
    assert torch.all((out - one).abs().float() <= 2.0 ** -7 * one.abs().float() + 2.0 ** -9)


@pytest.mark.parametrize("bs", [31, 128, 129, 700, 1024, 1025])
def test_many_sequences(bs):
    """Batches around the widths in which lengths are summed; most short or empty, some long, sharing a few pages."""
    rng = np.random.default_rng(bs)
    x = Inputs(40, [64 * 16], 2, 4, 64, 16, spare=1)
    pages = x.bt[0]
    x.lens = np.where(rng.random(bs) < 0.8, rng.integers(0, 40, bs), rng.integers(0, 4000, bs)).astype(np.int32)
    x.lens[-1] = 3333
    x.bt = pages[rng.integers(0, 64, (bs, 250))].astype(np.int32)
    x.q = torch.from_numpy(rng.standard_normal((bs, 1, 8, 64))).to(torch.bfloat16)
    rows = [(0, 0), (bs - 1, 7), (bs // 2, 3)] + [(int(b), 5) for b in rng.integers(0, bs, 8)]
    out, lse = x.run()
    x.check(out, lse, rows=rows)
    one, lse1 = x.run(num_splits=1)  # the same sums in another order: float32 and f16 roundings apart
    x.check(one, lse1, rows=rows)
    empty = torch.from_numpy(x.lens == 0).to(DEV)
    assert torch.all(out[empty] == 0) and torch.all(torch.isneginf(lse[empty]))
    live = ~empty
    assert torch.all((lse[live] - lse1[live]).abs() <= 2.0 ** -16)
    assert torch.all((out[live] - one[live]).abs().float() <= 2.0 ** -7 * one[live].abs().float() + 2.0 ** -9)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("bs,h_kv,q_len,group,mask,window,sinks", [
    (90, 8, 1, 3, False, 0, True), (170, 8, 1, 4, False, 20, False),
    (70, 9, 4, 4, True, 0, False), (200, 3, 2, 7, True, 9, True)])
def test_many_short_sequences(hd, bs, h_kv, q_len, group, mask, window, sinks):
    """More sequences than the GPU takes CTAs of four warps at once, of a few tiles each."""
    rng = np.random.default_rng(bs + hd)
    x = Inputs(400 + hd + bs, rng.integers(0, 70, bs), h_kv, group, hd, 16, q_len, mask, sinks)
    out, lse = x.run(window=window)
    x.check(out, lse, window=window, rows=[(int(b), int(h)) for b, h in zip(rng.integers(0, bs, 40),
                                                                           rng.integers(0, h_kv * group, 40))])
    one, lse1 = x.run(window=window, num_splits=1)  # the same sums in another order
    live = torch.isfinite(lse1)
    assert torch.equal(live, torch.isfinite(lse)) and torch.all((lse[live] - lse1[live]).abs() <= 2.0 ** -16)
    assert torch.all((out - one).abs().float() <= 2.0 ** -7 * one.abs().float() + 2.0 ** -9)


def test_bad_lengths_among_balanced_pieces():
    x = Inputs(50, [3000, 2000, 2500], 2, 4, 64, 16)
    good, good_lse = x.run()
    for n in (-1, 16 * x.bt.shape[1] + 1):
        x.lens[1] = n
        out, lse = x.run()
        assert fm.last_device_error() == fm.DEV_BAD_SEQLEN
        assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))
        assert torch.all((lse[[0, 2]] - good_lse[[0, 2]]).abs() <= 2.0 ** -16)


def test_offsets_past_32_bits():
    """Pages whose byte offsets pass 2^32 in codes and 2^29 in scales give what the same pages near the front do."""
    x = Inputs(51, [500, 130], 8, 4, 128, 16)
    want, want_lse = x.run()
    blocks = 620000  # 5.1 GB of codes a cache
    far = blocks - 1 - 7 * np.arange(x.codes[0].shape[0])
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    big = []
    for i in range(2):
        for small, width in ((x.codes[i], 64), (x.s8[i], 8)):
            t = torch.zeros((blocks, 8, 16, width), dtype=torch.uint8, device=DEV)
            t[torch.from_numpy(far).to(DEV)] = d(small)
            big.append(t)
    for splits in (0, 3):
        out, lse = fm.paged_gqa_decode_fp4(x.q.to(DEV), big[0], big[2], big[1], big[3], d(far[x.bt].astype(np.int32)),
                                           d(x.lens), torch.tensor([x.scale[0]], device=DEV),
                                           torch.tensor([x.scale[1]], device=DEV), softmax_scale=x.softmax_scale,
                                           num_splits=splits)
        torch.cuda.synchronize()
        assert torch.equal(out, want) or splits == 3
        x.check(out, lse)


def test_extreme_scores():
    """Scores that differ by hundreds, rising and falling along the keys: the reference moves often."""
    for sign in (1.0, -1.0):
        x = Inputs(10, [600, 700], 1, 4, 128, 16)
        x.q = (x.q * 40).to(torch.bfloat16)
        order = np.argsort(sign * (fp4.dequantise(x.codes[0], np.where(x.s8[0] & 0x7F == 0x7F, 0, x.s8[0]))
                                   [:, 0] @ x.q[0, 0, 0].double().numpy()).max(-1))
        x.bt[0, :37] = order[np.isin(order, x.bt[0, :37])]  # the first sequence's whole pages by their best key
        for splits in (1, 2):
            x.check(*x.run(num_splits=splits))


def test_queries_of_every_size():
    """Columns whose magnitudes differ by 2^80, a zero query, and one large value beside tiny ones."""
    x = Inputs(11, [500], 1, 8, 128, 16)
    for h, e in enumerate((-60, -20, 0, 3)):
        x.q[0, 0, h] = (x.q[0, 0, h].double() * 2.0 ** e).to(torch.bfloat16)
    x.q[0, 0, 4] = 0
    x.q[0, 0, 6] = (x.q[0, 0, 6].double() * 2.0 ** -133).to(torch.bfloat16)  # subnormal: scores of zero
    x.q[0, 0, 5] = x.q[0, 0, 5] * 2.0 ** -30
    x.q[0, 0, 5, 77] = 3.0
    x.check(*x.run())


def test_served_batch_sampled():
    """32 sequences of 1024 to 16384 keys and 8 KV heads, some (sequence, head) pairs against the oracle; page
    order and run to run bit-identical."""
    lens = np.random.default_rng(12).integers(1024, 16385, 32)
    rng = np.random.default_rng(13)
    x = Inputs(14, [16] * 1, 8, 4, 128, 16)  # a small pool, whose pages the batch shares
    pool = Inputs(15, [64 * 16], 8, 4, 128, 16, spare=1)
    x.codes, x.s8, x.scale = pool.codes, pool.s8, pool.scale
    x.lens = lens.astype(np.int32)
    pages = pool.bt[0]
    x.bt = pages[rng.integers(0, 64, (32, 1024))].astype(np.int32)
    x.q = torch.from_numpy(rng.standard_normal((32, 1, 32, 128))).to(torch.bfloat16)
    out, lse = x.run()
    x.check(out, lse, rows=[(0, 0), (3, 5), (31, 31), (17, 12), (8, 27)])
    again, lse2 = x.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    shift = np.roll(np.arange(x.codes[0].shape[0]), 7)  # block b moves to shift[b]
    for arr in (x.codes, x.s8):
        for i in range(2):
            moved = np.empty_like(arr[i])
            moved[shift] = arr[i]
            arr[i] = moved
    x.bt = shift[x.bt].astype(np.int32)
    moved, lse3 = x.run()
    assert torch.equal(out, moved) and torch.equal(lse, lse3)


@pytest.mark.parametrize("window", [33, 900])
@pytest.mark.parametrize("hd,q_len,group", [(64, 4, 2), (64, 4, 5), (128, 4, 2), (128, 6, 8), (256, 3, 2),
                                            (256, 16, 4)])
def test_a_nan_value_stays_with_the_tokens_that_see_it(hd, q_len, group, window):
    """A NaN V scale on the block's last key, which the last token alone sees, and on the key that the window leaves to
    the first token alone: those tokens' 16 dims are NaN and nothing else changes by a bit."""
    lens = [700, 40, 2000]
    x = Inputs(80 + hd + q_len, lens, 2, group, hd, 32, q_len)
    for splits in (0, 1, 2):
        want, want_lse = x.run(window=window, num_splits=splits)
        for b, n in enumerate(lens):
            first = n - q_len + 1 - window
            for j, tok, blk in [(n - 1, q_len - 1, hd // 16 - 1)] + ([(first, 0, 1)] if first >= 0 else []):
                at = x.bt[b, j // 32], 1, j % 32, blk
                kept = x.s8[1][at]
                x.s8[1][at] = 0xFF
                out, lse = x.run(window=window, num_splits=splits)
                x.s8[1][at] = kept
                touched = out[b, tok, group:, 16 * blk:16 * blk + 16]
                assert torch.all(torch.isnan(touched)), (splits, b, j)
                touched.copy_(want[b, tok, group:, 16 * blk:16 * blk + 16])
                assert torch.equal(out, want) and torch.equal(lse, want_lse), (splits, b, j)
    assert fm.last_device_error() == 0


@pytest.mark.parametrize("lens", [[50, 300, 20], [2000, 3000, 700], [900, 1300, 700]])
def test_nan_propagates_to_what_it_touches(lens):
    """A NaN query value: its row alone.  A NaN K scale on a visible key: every row of that KV head that sees it.  A NaN
    V scale: those rows' 16 dims alone, not the LSE.  Direct, cut, balanced and in clusters."""
    x = Inputs(70, lens, 2, 4, 128, 16)
    for splits in (0, 1, 2):
        want, want_lse = x.run(num_splits=splits)
        q = x.q.clone()
        x.q[1, 0, 2, 5] = math.nan
        out, lse = x.run(num_splits=splits)
        assert torch.all(torch.isnan(out[1, 0, 2])) and torch.isnan(lse[1, 0, 2])
        out[1, 0, 2], lse[1, 0, 2] = want[1, 0, 2], want_lse[1, 0, 2]
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        x.q = q
        page = x.bt[0, 2], 1, 3
        kept = x.s8[0][page].copy()
        x.s8[0][page] = 0x7F
        out, lse = x.run(num_splits=splits)
        assert torch.all(torch.isnan(out[0, 0, 4:])) and torch.all(torch.isnan(lse[0, 0, 4:]))
        out[0, 0, 4:], lse[0, 0, 4:] = want[0, 0, 4:], want_lse[0, 0, 4:]
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        x.s8[0][page] = kept
        kept = x.s8[1][page].copy()
        x.s8[1][page + (5,)] = 0x7F
        out, lse = x.run(num_splits=splits)
        assert torch.all(torch.isnan(out[0, 0, 4:, 80:96])) and torch.equal(lse, want_lse)
        out[0, 0, 4:, 80:96] = want[0, 0, 4:, 80:96]
        assert torch.equal(out, want)
        x.s8[1][page] = kept
    assert fm.last_device_error() == 0


def test_bad_pages_and_lengths_are_reported():
    x = Inputs(16, [100, 50], 1, 4, 64, 16)
    good, _ = x.run()
    x.bt[1, 2] = x.codes[0].shape[0]
    out, lse = x.run()
    assert fm.last_device_error() == fm.DEV_BAD_PAGE
    assert torch.equal(out[0], good[0])
    x.bt[1, 2] = -1
    x.run()
    assert fm.last_device_error() == fm.DEV_BAD_PAGE
    x.bt[1, 2] = 0
    for n in (-3, 16 * x.bt.shape[1] + 1):
        x.lens[1] = n
        out, lse = x.run()
        assert fm.last_device_error() == fm.DEV_BAD_SEQLEN
        assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))
        assert torch.equal(out[0], good[0])


def test_clusters_report_replay_and_overlap():
    """Errors of one sequence leave the others alone, entries past a sequence's end are not looked at; a captured call
    follows its lengths; two calls at once."""
    x = Inputs(19, [900, 400, 16], 2, 4, 128, 16)
    assert fm.gqa_fp4_workspace_bytes(3, 8, 2, 128, x.bt.shape[1] * 16) == 0
    good, good_lse = x.run()
    x.bt[1, 25:] = -7
    x.bt[2, 1:] = 1 << 30
    out, lse = x.run()
    assert fm.last_device_error() == 0 and torch.equal(out, good) and torch.equal(lse, good_lse)
    for page, entry in ((0, -1), (24, x.codes[0].shape[0])):
        kept, x.bt[1, page] = x.bt[1, page], entry
        out, _ = x.run()
        assert fm.last_device_error() == fm.DEV_BAD_PAGE
        assert torch.equal(out[[0, 2]], good[[0, 2]])
        x.bt[1, page] = kept
    for n in (-1, 16 * x.bt.shape[1] + 1):
        x.lens[0] = n
        out, lse = x.run()
        assert fm.last_device_error() == fm.DEV_BAD_SEQLEN
        assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[0])) and torch.equal(out[1:], good[1:])
    x.lens[0] = 900
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    t = dict(q=x.q.to(DEV), k_cache=d(x.codes[0]), v_cache=d(x.codes[1]), k_block_scales=d(x.s8[0]),
             v_block_scales=d(x.s8[1]), block_table=d(x.bt), seqlens=d(x.lens), softmax_scale=x.softmax_scale,
             k_scale=torch.tensor([x.scale[0]], device=DEV), v_scale=torch.tensor([x.scale[1]], device=DEV))
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            out, lse = torch.empty_like(good), torch.empty_like(good_lse)
            for _ in range(20):
                fm.paged_gqa_decode_fp4(**t, out=out, lse=lse)
            outs.append((out, lse))
    torch.cuda.synchronize()
    for out, lse in outs:
        assert torch.equal(out, good) and torch.equal(lse, good_lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fm.paged_gqa_decode_fp4(**t, out=out, lse=lse)
        fm.paged_gqa_decode_fp4(**t, out=out, lse=lse)
    for lens in ([17, 0, 3], [890, 399, 1]):
        t["seqlens"].copy_(torch.tensor(lens, dtype=torch.int32))
        x.lens = np.asarray(lens, np.int32)
        g.replay()
        torch.cuda.synchronize()
        x.check(out, lse)


def test_outputs_given_graph_and_two_streams():
    """Own outputs and workspaces, a captured call replayed with new lengths, two calls at once."""
    x = Inputs(17, [900, 400, 16], 2, 4, 128, 16)
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    t = dict(q=x.q.to(DEV), k_cache=d(x.codes[0]), v_cache=d(x.codes[1]), k_block_scales=d(x.s8[0]),
             v_block_scales=d(x.s8[1]), block_table=d(x.bt), seqlens=d(x.lens),
             k_scale=torch.tensor([x.scale[0]], device=DEV), v_scale=torch.tensor([x.scale[1]], device=DEV))
    want, want_lse = fm.paged_gqa_decode_fp4(**t, num_splits=4)
    out3, _ = fm.paged_gqa_decode_fp4(**{**t, "q": t["q"][:, 0].contiguous()}, num_splits=4)
    assert out3.shape == (3, 8, 128) and torch.equal(out3, want[:, 0])
    need = fm.gqa_fp4_workspace_bytes(3, 8, 2, 128, x.bt.shape[1] * 16, num_splits=4)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            out, lse = torch.empty_like(want), torch.empty_like(want_lse)
            ws = torch.empty(need, dtype=torch.uint8, device=DEV)
            for _ in range(20):
                fm.paged_gqa_decode_fp4(**t, num_splits=4, out=out, lse=lse, workspace=ws)
            outs.append((out, lse, ws))
    torch.cuda.synchronize()
    for out, lse, _ in outs:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    out, lse, ws = outs[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fm.paged_gqa_decode_fp4(**t, num_splits=4, out=out, lse=lse, workspace=ws)
        fm.paged_gqa_decode_fp4(**t, num_splits=4, out=out, lse=lse, workspace=ws)
    t["seqlens"] -= 10
    g.replay()
    torch.cuda.synchronize()
    want, want_lse = fm.paged_gqa_decode_fp4(**t, num_splits=4)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    none, _ = fm.paged_gqa_decode_fp4(**{**t, "q": t["q"][:0], "block_table": t["block_table"][:0],
                                        "seqlens": t["seqlens"][:0]})
    assert none.shape == (0, 1, 8, 128)
    assert fm.last_device_error() == 0


def test_wrapper_refusals():
    x = Inputs(18, [20], 1, 4, 128, 16)
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    ok = dict(q=x.q.to(DEV), k_cache=d(x.codes[0]), v_cache=d(x.codes[1]), k_block_scales=d(x.s8[0]),
              v_block_scales=d(x.s8[1]), block_table=d(x.bt), seqlens=d(x.lens),
              k_scale=torch.tensor([x.scale[0]], device=DEV), v_scale=torch.tensor([x.scale[1]], device=DEV))
    for bad in [dict(q=ok["q"].float()), dict(q=ok["q"].cpu()), dict(q=ok["q"][..., :64]),
                dict(v_cache=ok["v_cache"][:1]), dict(k_block_scales=ok["k_block_scales"][..., :4]),
                dict(k_block_scales=ok["k_block_scales"].float()), dict(v_scale=None),
                dict(block_table=ok["block_table"].long()), dict(seqlens=ok["seqlens"].cpu()),
                dict(spec_mask=torch.zeros((1, 2, 2), dtype=torch.uint8, device=DEV)),
                dict(sinks=torch.zeros(3, device=DEV)), dict(out=ok["q"].float()),
                dict(lse=torch.zeros((1, 1, 5), device=DEV))]:
        with pytest.raises(ValueError):
            fm.paged_gqa_decode_fp4(**{**ok, **bad})
    with pytest.raises(fm.FP8MLAError) as err:
        fm.paged_gqa_decode_fp4(**{**ok, "k_cache": ok["k_cache"].view(torch.float8_e4m3fn),
                                   "v_cache": ok["v_cache"].view(torch.float8_e4m3fn)})
    assert err.value.status == 2
    for bad in (dict(softmax_scale=0.0), dict(window=-1), dict(num_splits=-1)):
        with pytest.raises(fm.FP8MLAError):
            fm.paged_gqa_decode_fp4(**{**ok, **bad})
