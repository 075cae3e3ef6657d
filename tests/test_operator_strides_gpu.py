"""A dimension of one element has no stride that matters: single tokens and single heads out of wider buffers."""

import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
HD = 64


def _caches(h_kv):
    return [torch.zeros((2, h_kv, 16, HD), dtype=torch.uint8, device=DEV) for _ in range(2)]


@pytest.mark.parametrize("n,h_kv,h_q,strides", [(1, 2, 4, (1001, HD)), (3, 1, 1, (3 * HD, 5)), (1, 1, 1, (1, 3)),
                                                (1, 2, 1, (7, HD))])
def test_odd_strides_of_single_elements(n, h_kv, h_q, strides):
    g = torch.Generator().manual_seed(1)
    buf = [torch.randn(2048, generator=g).to(torch.bfloat16).to(DEV) for _ in range(3)]
    k, v = (b.as_strided((n, h_kv, HD), strides + (1,)) for b in buf[:2])
    q = buf[2].as_strided((n, h_q, HD), strides + (1,))
    f, _ = fm.rotary_frequencies(HD)
    table, pos = fm.rotary_table(f, 32), torch.arange(7, 7 + n, device=DEV)
    slots, one = torch.arange(n, dtype=torch.int32, device=DEV), torch.ones(1, device=DEV)
    kw = dict(positions=pos, table=table, k_scale=one, v_scale=one)
    a, b = _caches(h_kv), _caches(h_kv)
    k1, v1, q1 = (torch.empty(t.shape, dtype=t.dtype, device=DEV).copy_(t) for t in (k, v, q))
    want = fm.paged_kv_append(k1, v1, slots, *a, **kw, q=q1)
    got = fm.paged_kv_append(k, v, slots, *b, **kw, q=q)
    assert torch.equal(got, want) and all(torch.equal(x, y) for x, y in zip(a, b))
    turned, turned_k = fm.rotary_apply(q, k, pos, table)
    assert torch.equal(turned, want)
    out = torch.zeros(2048, dtype=torch.bfloat16, device=DEV).as_strided((n, h_kv, HD), strides + (1,))
    fm.rotary_apply(k, None, pos, table, q_out=out)
    assert torch.equal(out, turned_k)
    fm.rotary_apply(k, None, pos, table, q_out=k)
    assert torch.equal(k, turned_k) and fm.last_device_error() == 0
