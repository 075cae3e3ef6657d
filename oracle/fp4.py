"""CPU oracle for the 4-bit cache: E2M1 codes, block scales, append and decode.

TEST INFRASTRUCTURE ONLY, under the same rule as ``oracle.attention``.

value = scale * E4M3(s8) * E2M1(code), one s8 per 16 values of a row, codes
two to a byte with the even dimension in the low nibble.  Quantisation is
decided in float32 with round-to-nearest-even operations, like the E4M3
cache write: s8 = E4M3(fp32(amax * fp32(1 / fp32(6 scale)))), code =
E2M1(fp32(x * fp32(1 / fp32(s8 scale)))), 0 where s8 is 0.
"""

from __future__ import annotations

import math

import numpy as np

from .attention import as_bytes, as_float64, as_int64, e4m3_decode, softmax_attention, spec_visible
from .cache_write import e4m3_encode

BLOCK = 16


def e2m1_value(code: int) -> float:
    """Value of one 4-bit code: sign, 2-bit exponent with bias 1, 1-bit mantissa, no infinity or NaN."""
    sign = -1.0 if code & 8 else 1.0
    exponent, mantissa = (code >> 1) & 3, code & 1
    if exponent == 0:
        return sign * mantissa * 0.5
    return sign * (1.0 + mantissa / 2.0) * 2.0 ** (exponent - 1)


E2M1_TABLE = np.array([e2m1_value(c) for c in range(16)], dtype=np.float64)


def e2m1_encode(y) -> np.ndarray:
    """Codes of the nearest values, ties to the even code, magnitudes above 6 saturate; the sign is kept."""
    y = np.asarray(y, dtype=np.float64)
    if not np.all(np.isfinite(y)):
        raise ValueError("e2m1_encode: non-finite input")
    mags = E2M1_TABLE[:8]
    d = np.abs(np.abs(y)[..., None] - mags)
    best = d.min(axis=-1, keepdims=True)
    # among equally near codes the even one
    cand = np.where(d == best, np.arange(8), 99)
    odd_last = np.where(cand % 2 == 0, cand, cand + 50)
    code = odd_last.min(axis=-1)
    code = np.where(code >= 50, code - 50, code)
    return (code | (np.signbit(y).astype(np.int64) << 3)).astype(np.uint8)


def quantise(x, scale: float):
    """(packed codes [..., hd / 2], s8 codes [..., hd / 16]) of x [..., hd] (float32 values)."""
    x = np.asarray(as_float64(x), dtype=np.float32)
    g = np.float32(scale)
    blocks = x.reshape(*x.shape[:-1], -1, BLOCK)
    amax = np.abs(blocks).max(axis=-1)
    inv6 = np.float32(1.0) / np.float32(g * np.float32(6.0))
    s8 = e4m3_encode((amax * inv6).astype(np.float32))
    s = e4m3_decode(s8).astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(s > 0, np.float32(1.0) / (s * g).astype(np.float32), np.float32(0.0)).astype(np.float32)
    y = (blocks * inv[..., None]).astype(np.float32)
    codes = np.where((s > 0)[..., None], e2m1_encode(y), 0).astype(np.uint8)
    codes = codes.reshape(x.shape)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), s8


def dequantise(codes, s8, scale: float = 1.0) -> np.ndarray:
    """float64 values [..., hd] of packed codes [..., hd / 2] and block scales [..., hd / 16]."""
    codes, s8 = as_bytes(codes), as_bytes(s8)
    e = np.empty((*codes.shape[:-1], codes.shape[-1] * 2))
    e[..., 0::2] = E2M1_TABLE[codes & 15]
    e[..., 1::2] = E2M1_TABLE[codes >> 4]
    return e * np.repeat(e4m3_decode(s8), BLOCK, axis=-1) * float(scale)


def gqa_decode(q, k_cache, v_cache, k_s8, v_s8, block_table, seqlens, k_scale, v_scale, softmax_scale,
               spec_mask=None, window: int = 0, sinks=None, rows=None):
    """Paged GQA decode over a 4-bit cache in float64, with the options of
    ``oracle.attention.gqa_decode_ext``.  q [bs, q_len, h_q, hd].  Returns (out, lse, weight) where
    weight[b, i, h] = sum_j p_j |v_j| per dim, what a rounding of the probabilities is measured by.
    ``rows`` restricts the work to some (sequence, query head) pairs (others stay 0 / NaN)."""
    q = as_float64(q)
    kc, vc = as_bytes(k_cache), as_bytes(v_cache)
    ks, vs = as_bytes(k_s8), as_bytes(v_s8)
    bt, sl = as_int64(block_table), as_int64(seqlens)
    bs, q_len, h_q, hd = q.shape
    h_kv, page = kc.shape[1], kc.shape[2]
    group = h_q // h_kv
    sk = None if sinks is None else as_float64(sinks)
    out = np.zeros((bs, q_len, h_q, hd))
    weight = np.zeros((bs, q_len, h_q, hd))
    lse = np.full((bs, q_len, h_q), np.nan)
    todo = rows if rows is not None else [(b, h) for b in range(bs) for h in range(h_q)]
    kept = {}
    for bi, h in todo:
        s_k, kvh = int(sl[bi]), h // group
        if (bi, kvh) not in kept:
            pages = [int(bt[bi, p]) for p in range((s_k + page - 1) // page)]
            if pages:
                keys = np.concatenate([dequantise(kc[p, kvh], ks[p, kvh], k_scale) for p in pages])[:s_k]
                vals = np.concatenate([dequantise(vc[p, kvh], vs[p, kvh], v_scale) for p in pages])[:s_k]
            else:
                keys = vals = np.zeros((0, hd))
            kept = {(bi, kvh): (keys, vals)}
        keys, vals = kept[(bi, kvh)]
        for i in range(q_len):
            vis = spec_visible(s_k, q_len, i, None if spec_mask is None else as_int64(spec_mask)[bi, i], window)
            score = (keys[vis] @ q[bi, i, h]) * float(softmax_scale)
            o, l = softmax_attention(score, vals[vis])
            a, _ = softmax_attention(score, np.abs(vals[vis]))
            if sk is not None and sk[h] != -math.inf:
                m = max(l, sk[h])
                w = math.exp(l - m) if l != -math.inf else 0.0
                total = w + math.exp(sk[h] - m)
                o, a, l = o * (w / total), a * (w / total), m + math.log(total)
            out[bi, i, h], weight[bi, i, h], lse[bi, i, h] = o, a, l
    return out, lse, weight
