"""Cross attention, shared prefixes and merges where offsets pass 32 bits: caches, queries and outputs of more than 4 GB."""

import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("rows", [False, True])
def test_pages_past_4_gb(rows):
    """Pages at the end of a cache of 2^32 bytes and more give what the same pages give in a small one."""
    h_kv, page, hd, few = 8, 16, 128, 12
    far = (1 << 32) // (h_kv * page * hd) + 5
    gen = torch.Generator(device=DEV).manual_seed(3)
    small = [torch.randn(few, h_kv, page, hd, generator=gen, device=DEV).to(torch.float8_e4m3fn) for _ in range(2)]
    scale = [torch.rand(few, h_kv, page, generator=gen, device=DEV) + 0.5 for _ in range(2)]
    large = [torch.empty((far + few, h_kv, page, hd), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    large_scale = [torch.empty((far + few, h_kv, page), device=DEV) for _ in range(2)]
    for a, b in zip(large + large_scale, small + scale):
        a[far:].copy_(b)
    one = torch.ones(1, device=DEV)
    s, ls = (scale, large_scale) if rows else ((one, one), (one, one))
    q = torch.randn(6, 3, 32, hd, generator=gen, device=DEV).to(torch.bfloat16)
    prefix, own = _i32(7, 2, 9, 0)[None], _i32(1, 3, 4, 5, 6, 8, 10, 11, 1, 3, 4, 5).reshape(6, 2)
    lens = _i32(32, 3, 17, 0, 20, 5)

    def calls(k, v, ks, vs, first):
        yield fm.paged_cross_attention(q[:, 0], k, v, own + first, lens, ks, vs)
        yield fm.paged_cross_attention(q.reshape(18, 32, hd), k, v, prefix + first, _i32(57), ks, vs, q_starts=_i32(0, 18))
        yield fm.paged_gqa_decode_shared(q, k, v, prefix + first, _i32(57), _i32(0, 5), own + first, lens, ks, vs)

    for near, away in zip(calls(*small, *s, 0), calls(*large, *ls, far)):
        assert torch.equal(near[0], away[0]) and torch.equal(near[1], away[1])
    assert fm.last_device_error() == 0


def test_queries_past_4_gb():
    """The last tokens of queries and outputs of more than 2^31 values, behind a sequence that has the others."""
    tokens, h_q, hd, tail = (1 << 31) // (32 * 128) + 300, 32, 128, 130
    gen = torch.Generator(device=DEV).manual_seed(4)
    k, v = (torch.randn(4, 8, 16, hd, generator=gen, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    q = torch.zeros((tokens, h_q, hd), dtype=torch.bfloat16, device=DEV)
    q[-tail:].copy_(torch.randn(tail, h_q, hd, generator=gen, device=DEV))
    one, table = torch.ones(1, device=DEV), _i32(2, 0, 3, 1).reshape(2, 2)
    out, lse = fm.paged_cross_attention(q, k, v, table, _i32(20, 31), one, one,
                                        q_starts=_i32(0, tokens - tail, tokens))
    want = fm.paged_cross_attention(q[-tail:].contiguous(), k, v, table[1:].contiguous(), _i32(31), one, one,
                                    q_starts=_i32(0, tail))
    assert torch.equal(out[-tail:], want[0]) and torch.equal(lse[-tail:], want[1])
    # queries of zeros: the mean of the keys' values (f16 weights that are equal; bf16's rounding and float32 sums)
    mean = torch.cat((v[2], v[0]), 1)[:, :20].double().mean(1).repeat_interleave(4, 0)
    for t in (0, tokens // 2, tokens - tail - 1):
        assert bool(((out[t].double() - mean).abs() <= 2.0 ** -8 * mean.abs() + 2.0 ** -20).all())
    assert fm.last_device_error() == 0


def test_merges_past_4_gb():
    tokens, heads, dim, tail = (1 << 31) // (32 * 128) + 77, 32, 128, 90
    gen = torch.Generator(device=DEV).manual_seed(6)
    outs, lses, ends = [], [], []
    for _ in range(2):
        end = torch.randn(tail, heads, dim, generator=gen, device=DEV).to(torch.bfloat16)
        x = torch.zeros((tokens, heads, dim), dtype=torch.bfloat16, device=DEV)
        l = torch.randn(tokens, heads, generator=gen, device=DEV)
        x[-tail:].copy_(end)
        outs.append(x), lses.append(l), ends.append(end)
    out, lse = fm.attention_merge(outs, lses)
    want = fm.attention_merge(ends, [l[-tail:].contiguous() for l in lses])
    assert torch.equal(out[-tail:], want[0]) and torch.equal(lse[-tail:], want[1])
    assert not bool(out[:-tail].any())
