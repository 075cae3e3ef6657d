"""CPU oracle of cross attention, decode behind shared prefixes and the merge of partial results.

TEST INFRASTRUCTURE ONLY, under the same rule as ``oracle.attention``.

Everything is float64.  ``attend`` also returns what the tolerances of the GPU
tests are made of: sum p |v| and the largest |v| of every output row, and the
largest size of the terms of a row's scores.
"""

from __future__ import annotations

import numpy as np

from .attention import as_bytes, as_float64, as_int64, e4m3_decode, spec_visible


def gather(cache, scale, table_row, keys: int, head: int) -> np.ndarray:
    """[keys, head_dim] of one KV head: codes times the cache's scale, or their row's."""
    codes = as_bytes(cache)
    page = codes.shape[2]
    pages = as_int64(table_row)[:-(-keys // page)]
    rows = e4m3_decode(codes[pages, head]).reshape(-1, codes.shape[3])[:keys]
    scale = np.asarray(as_float64(scale))
    if scale.size == 1:
        return rows * scale.reshape(-1)[0]
    return rows * scale[pages, head].reshape(-1)[:keys, None]


def attend(q, k, v, softmax_scale: float, visible=None, sink=None):
    """One row q [hd] to k, v [keys, hd]: (out, lse, sum p |v|, largest |v|, largest sum of |terms| of a score)."""
    hd = q.shape[0]
    s = (k @ q) * softmax_scale
    # a term is taken with a quarter of the row's largest query beside its own: see the GPU tests' tolerance
    size = (np.abs(k) @ (np.abs(q) + np.abs(q).max() / 4)).max() * softmax_scale if len(s) else 0.0
    if visible is not None:
        s = np.where(visible, s, -np.inf)
    everything = s if sink is None else np.append(s, sink)
    top = everything.max() if everything.size else -np.inf
    if top == -np.inf:
        return np.zeros(hd), -np.inf, np.zeros(hd), np.zeros(hd), size
    p = np.exp(everything - top)
    total = p.sum()
    p = p[:len(s)] / total
    if visible is not None:  # what a hidden key holds does not count
        v = np.where(visible[:, None], v, 0.0)
    return p @ v, top + np.log(total), p @ np.abs(v), np.abs(v).max(0, initial=0.0), size


def _rows(n, heads, hd):
    return (np.zeros((n, heads, hd)), np.full((n, heads), -np.inf), np.zeros((n, heads, hd)), np.zeros((n, heads, hd)),
            np.zeros((n, heads)))


def cross(q, k_cache, v_cache, table, kv_lens, k_scale, v_scale, softmax_scale, starts=None):
    """(out, lse, sum p |v|, largest |v|, sizes) of every token; tokens of no sequence as of one without keys."""
    q = as_float64(q)
    n, heads, hd = q.shape
    h_kv = k_cache.shape[1]
    group = heads // h_kv
    lens = as_int64(kv_lens)
    starts = np.arange(len(lens) + 1) if starts is None else as_int64(starts)
    res = _rows(n, heads, hd)
    for b, keys in enumerate(lens):
        for h in range(h_kv):
            k = gather(k_cache, k_scale, table[b], keys, h)
            v = gather(v_cache, v_scale, table[b], keys, h)
            for t in range(starts[b], starts[b + 1]):
                for x in range(h * group, (h + 1) * group):
                    for r, value in zip(res, attend(q[t, x], k, v, softmax_scale)):
                        r[t, x] = value
    return res


def shared(q, k_cache, v_cache, prefix_table, prefix_lens, prefix_starts, table, lens, k_scale, v_scale, softmax_scale,
           mask=None, sinks=None):
    """The same for q [bs, q_len, heads, hd], as if every sequence had its prefix to itself."""
    q = as_float64(q)
    bs, q_len, heads, hd = q.shape
    h_kv = k_cache.shape[1]
    group = heads // h_kv
    lens, prefix_lens, starts = as_int64(lens), as_int64(prefix_lens), as_int64(prefix_starts)
    res = _rows(bs * q_len, heads, hd)
    for b in range(bs):
        mine = [g for g in range(len(prefix_lens)) if starts[g] <= b < starts[g + 1]]
        for h in range(h_kv):
            k = gather(k_cache, k_scale, table[b], lens[b], h)
            v = gather(v_cache, v_scale, table[b], lens[b], h)
            front = 0
            for g in mine:
                front = prefix_lens[g]
                k = np.concatenate((gather(k_cache, k_scale, prefix_table[g], front, h), k))
                v = np.concatenate((gather(v_cache, v_scale, prefix_table[g], front, h), v))
            for i in range(q_len):
                own = spec_visible(int(lens[b]), q_len, i, None if mask is None else np.asarray(mask)[b, i]) \
                    if q_len > 1 or mask is not None else np.ones(lens[b], bool)
                visible = np.concatenate((np.ones(front, bool), own))
                for x in range(h * group, (h + 1) * group):
                    sink = None if sinks is None else float(as_float64(sinks)[x])
                    for r, value in zip(res, attend(q[b, i, x], k, v, softmax_scale, visible, sink)):
                        r[b * q_len + i, x] = value
    return res


def merge(outs, lses):
    """(out, lse) of results over disjoint keys."""
    lse = np.stack([as_float64(x) for x in lses])
    top = lse.max(0)
    base = np.where(top == -np.inf, 0.0, top)
    w = np.exp(lse - base)
    total = w.sum(0)
    part = np.stack([np.where((x == -np.inf)[..., None], 0.0, as_float64(o)) for o, x in zip(outs, lse)])
    out = np.divide((part * w[..., None]).sum(0), total[..., None], where=total[..., None] > 0,
                    out=np.zeros(part.shape[1:]))
    with np.errstate(divide="ignore"):
        return out, base + np.log(total)
