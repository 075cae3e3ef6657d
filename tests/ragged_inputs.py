"""Seeded inputs and tolerances of the tests of cross attention and shared prefixes."""

import math

import numpy as np
import torch

from oracle import ragged
from oracle.cache_write import e4m3_encode


def tolerance(want, keys):
    """(of out, of lse) for (out, lse, sum p |v|, largest |v|, sizes) of the oracle, before any run.

    Scores: K enters exactly; Q, scaled to 448 at most, as two E4M3 terms, which are off by 2^-10 at most, 2^-18 of the
    row's largest value (they are exact from 2^-10 of it on), or as it is; a product of head_dim <= 128 terms (twice,
    with two of Q) is summed in float32, 256 roundings of 2^-24 at most.  With size = scale sum |k| (|q| + largest / 4)
    that is 2^-16 size for both.  LSE: no more than that, the approximate 2^x and log2 and float32 sums (2^-20) and the
    roundings of the reference and the result (2^-22 of their size).  Outputs: a weight is off by the f16 rounding 2^-11,
    twice the score's error (its own and the sum's) and 2^-20, against sum p |v|; then the rounding to bf16, 2^-8 of the
    value.  f16's spacing below its normal numbers is 2^-24 where the largest weight is 2^7 or more: keys * 2^-32 of the
    largest |v|."""
    out, lse, pv, most, size = want
    e = 2.0 ** -16 * size
    finite = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    tol_lse = e + 2.0 ** -20 + 2.0 ** -22 * (finite + size)
    tol_out = 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2 * e[..., None] + 2.0 ** -20) * pv + keys * 2.0 ** -32 * most
    return tol_out, tol_lse


def within(got_out, got_lse, want, keys):
    """The first thing that is wrong, or None."""
    out, lse = got_out.double().cpu().numpy().reshape(want[0].shape), got_lse.double().cpu().numpy().reshape(want[1].shape)
    tol_out, tol_lse = tolerance(want, keys)
    empty = want[1] == -np.inf
    if not np.array_equal(lse == -np.inf, empty):
        return "rows without keys"
    if not np.all(out[empty] == 0):
        return "rows without keys are not zero"
    bad = ~(np.abs(out - want[0]) <= tol_out)
    if bad.any():
        return f"out: {bad.sum()} of {bad.size}, worst {np.max(np.abs(out - want[0]) / np.maximum(tol_out, 1e-30)):.2f} of the tolerance"
    with np.errstate(invalid="ignore"):
        bad = ~(empty | (np.abs(lse - want[1]) <= tol_lse))
    if bad.any():
        return f"lse: {bad.sum()} of {bad.size}"
    return None


class Pool:
    """Caches whose pages are handed out in random order; what no key owns holds NaN codes (and NaN row scales)."""

    def __init__(self, seed, lens_of, h_kv, hd, page, rows, spare=3):
        self.rng = rng = np.random.default_rng(seed)
        self.h_kv, self.hd, self.page, self.by_row = h_kv, hd, page, rows
        counts = [[-(-int(n) // page) for n in lens] for lens in lens_of]
        total = sum(map(sum, counts)) + spare
        perm = rng.permutation(total)
        x = [rng.standard_normal((total, h_kv, page, hd)) * np.exp(0.4 * rng.standard_normal(hd)) for _ in range(2)]
        if rows:
            x = [a * rng.uniform(0.25, 2.0, (total, h_kv, page, 1)) for a in x]
        owned = np.zeros((total, page), bool)
        self.tables, at = [], 0
        for lens, count in zip(lens_of, counts):
            t = np.full((len(lens), max([1, *count])), perm[-1], np.int32)
            for i, (n, c) in enumerate(zip(lens, count)):
                t[i, :c] = perm[at:at + c]
                for j in range(c):
                    owned[perm[at + j], :min(page, int(n) - j * page)] = True
                at += c
            self.tables.append(t)
        self.cache, self.scale = [], []
        for a in x:
            s = np.abs(a).max(-1) / 448 if rows else np.array([np.abs(a).max() / 448])
            s = s.astype(np.float32)
            codes = e4m3_encode(a / (s[..., None] if rows else s))
            hole = np.broadcast_to(~owned[:, None], codes.shape[:3])
            codes[hole] = np.where(rng.random((int(hole.sum()), hd)) < 0.5, 0x7F, 0xFF)
            if rows:
                s[hole] = np.nan
            self.cache.append(codes), self.scale.append(s)
        self.softmax_scale = float(np.float32(1 / math.sqrt(hd)))

    def queries(self, *shape, size=1.0):
        return (torch.from_numpy(self.rng.standard_normal((*shape, self.hd)) * size)).to(torch.bfloat16)

    def device(self, dev):
        d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)  # noqa: E731
        return [d(self.cache[0]).view(torch.float8_e4m3fn), d(self.cache[1]).view(torch.float8_e4m3fn),
                *[d(t) for t in self.tables], d(self.scale[0]), d(self.scale[1])]


def cross_case(seed, q_lens, kv_lens, h_kv, group, hd, page, rows, pad=(0, 0), size=1.0):
    """(pool, q, starts, want) of a ragged batch; pad: tokens of no sequence in front and behind."""
    pool = Pool(seed, [kv_lens], h_kv, hd, page, rows)
    starts = np.concatenate(([0], np.cumsum(q_lens))).astype(np.int32) + pad[0]
    q = pool.queries(int(starts[-1]) + pad[1], h_kv * group, size=size)
    want = ragged.cross(q, *pool.cache, pool.tables[0], kv_lens, *pool.scale, pool.softmax_scale, starts)
    return pool, q, starts, want


def shared_case(seed, prefix_lens, prefix_starts, lens, h_kv, group, hd, page, rows, q_len=1, mask=False, sinks=False):
    pool = Pool(seed, [prefix_lens, lens], h_kv, hd, page, rows)
    q = pool.queries(len(lens), q_len, h_kv * group)
    m = (pool.rng.random((len(lens), q_len, q_len)) < 0.5).astype(np.uint8) if mask else None
    s = pool.rng.standard_normal(h_kv * group).astype(np.float32) if sinks else None
    want = ragged.shared(q, *pool.cache, pool.tables[0], prefix_lens, prefix_starts, pool.tables[1], lens, *pool.scale,
                         pool.softmax_scale, m, s)
    return pool, q, m, s, want
