"""Outputs of the rotary, append, read-back and 4-bit decode calls: in place, between each other's rows, or refused."""

import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from tests.test_gqa_fp4_gpu import Inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _rows(*shape):
    g = torch.Generator().manual_seed(3)
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)


def _table(rot, n=64):
    f, _ = fm.rotary_frequencies(rot)
    return fm.rotary_table(f, n)


@pytest.mark.parametrize("order", ["tokens", "heads", "dims"])
def test_rotation_between_each_others_rows(order):
    """Queries and keys of one projection turned in place, and into another buffer of its layout."""
    n, hq, hk, hd = 9, 6, 2, 64
    pos, table = torch.arange(n, device=DEV), _table(hd)

    def split(x):
        if order == "tokens":   # [n, heads, hd]
            return x[:, :hq], x[:, hq:hq + hk]
        if order == "heads":    # [heads, n, hd]
            x = x.reshape(hq + 2 * hk, n, hd).transpose(0, 1)
            return x[:, :hq], x[:, hq:hq + hk]
        x = x.reshape(n, -1, 2 * hd)  # a query head beside another tensor's
        return x[:, :, :hd], x[:, :, hd:]

    x, y = _rows(n, hq + 2 * hk, hd), torch.zeros((n, hq + 2 * hk, hd), dtype=torch.bfloat16, device=DEV)
    q, k = split(x)
    want = [t.clone() for t in fm.rotary_apply(q, k, pos, table)]
    fm.rotary_apply(q, k, pos, table, q_out=split(y)[0], k_out=split(y)[1])
    assert torch.equal(split(y)[0], want[0]) and torch.equal(split(y)[1], want[1])
    fm.rotary_apply(q, k, pos, table, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_rotation_refusals():
    pos, table = torch.arange(4, device=DEV), _table(32)
    x, buf = _rows(4, 6, 32), torch.zeros(2000, dtype=torch.bfloat16, device=DEV)
    q, k = x[:, :4], x[:, 4:]
    for q_out, k_out in [(buf.as_strided((4, 4, 32), (64, 16, 1)), None),
                         (buf.as_strided((4, 4, 32), (32, 32, 1)), None),
                         (buf[:512].view(4, 4, 32), buf[256:512].view(4, 2, 32)), (x[:, 1:5], None), (None, x[:, 3:5]),
                         (x.view(-1)[:512].view(4, 4, 32), None)]:
        with pytest.raises(fm.FP8MLAError):
            fm.rotary_apply(q, k, pos, table, q_out=q_out, k_out=k_out)


def test_append_in_the_queries_place_and_refusals():
    n, shape = 7, (4, 2, 16, 32)
    q, kv = _rows(n, 4, 64), _rows(n, 4, 64)
    slots, pos, table = (torch.arange(n, dtype=torch.int32, device=DEV), torch.arange(n, device=DEV), _table(64))
    scale = torch.tensor([0.002], device=DEV)

    def caches():
        return dict(k_cache=torch.zeros(shape, dtype=torch.uint8, device=DEV),
                    v_cache=torch.zeros(shape, dtype=torch.uint8, device=DEV),
                    k_block_scales=torch.zeros(shape[:3] + (4,), dtype=torch.uint8, device=DEV),
                    v_block_scales=torch.zeros(shape[:3] + (4,), dtype=torch.uint8, device=DEV))

    def call(q, c, **kw):
        return fm.paged_kv_append(kv[:, :2], kv[:, 2:], slots, **c, positions=pos, table=table, k_scale=scale,
                                  v_scale=scale, q=q, **kw)

    a, b = caches(), caches()
    want, mine = call(q, a), q.clone()
    assert call(mine, b, q_out=mine) is mine
    assert torch.equal(mine, want) and all(torch.equal(a[x], b[x]) for x in a)
    for bad in (dict(a, v_cache=a["k_cache"]), dict(a, v_block_scales=a["k_block_scales"])):
        with pytest.raises(fm.FP8MLAError):
            call(q, bad)
    with pytest.raises(fm.FP8MLAError):
        call(q, a, q_out=kv)  # over keys and values
    with pytest.raises(fm.FP8MLAError):
        fm.paged_cache_read(a["k_cache"], slots, scale=scale, block_scales=a["k_block_scales"],
                            out=a["k_cache"].view(-1)[:n * 256].view(torch.bfloat16).view(n, 2, 64))


@pytest.mark.parametrize("lens,h_kv,group,hd,splits", [
    ([300, 0, 17], 2, 4, 128, 0), ([900], 2, 4, 128, 0), ([300, 40], 2, 12, 64, 1), ([900, 300], 2, 4, 256, 3),
    ([9001, 4000], 1, 4, 128, 0), ([100] * 240, 2, 4, 64, 0)])
def test_attention_in_the_queries_place(lens, h_kv, group, hd, splits):
    x = Inputs(30, lens, h_kv, group, hd, 16)
    want, want_lse = x.run(num_splits=splits)
    d = lambda t: torch.from_numpy(t).to(DEV)  # noqa: E731
    q = x.q.to(DEV)
    out, lse = fm.paged_gqa_decode_fp4(q, d(x.codes[0]), d(x.codes[1]), d(x.s8[0]), d(x.s8[1]), d(x.bt), d(x.lens),
                                       torch.tensor([x.scale[0]], device=DEV), torch.tensor([x.scale[1]], device=DEV),
                                       softmax_scale=x.softmax_scale, num_splits=splits, out=q)
    assert out is q and torch.equal(out, want) and torch.equal(lse, want_lse)
    with pytest.raises(fm.FP8MLAError):
        fm.paged_gqa_decode_fp4(q, d(x.codes[0]), d(x.codes[1]), d(x.s8[0]), d(x.s8[1]), d(x.bt), d(x.lens),
                                torch.tensor([x.scale[0]], device=DEV), torch.tensor([x.scale[1]], device=DEV),
                                lse=q.view(-1)[:2 * lse.numel()].view(torch.float32).view(lse.shape))
    assert fm.last_device_error() == 0
