"""Outputs of cross attention and shared prefixes beside their inputs in one block of memory, and on them."""

import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def test_beside_and_on_the_inputs():
    hd, h, page, blocks, n = 64, 2, 16, 4, 3
    cache, row = blocks * h * page * hd, n * h * hd * 2
    buf = torch.zeros(256 + 2 * cache + 2 * row + 1024, dtype=torch.uint8, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(1)
    k, v = (buf[256 + i * cache:][:cache].view(torch.float8_e4m3fn).view(blocks, h, page, hd) for i in range(2))
    for x in (k, v):
        x.copy_(torch.randn(x.shape, generator=gen, device=DEV).to(torch.float8_e4m3fn))
    q = torch.randn(n, h, hd, generator=gen, device=DEV).to(torch.bfloat16)
    one = torch.ones(1, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    table, lens = i32(2, 0, 1, 3, 3, 1).view(3, 2), i32(20, 32, 5)
    args = (q, k, v, table, lens, one, one)
    shared = (q, k, v, table[:1], lens[:1], i32(0, 2), table, lens, one, one)
    end = 256 + 2 * cache
    beside = buf[end:end + row].view(torch.bfloat16).view(n, h, hd), buf[end + row:end + row + n * h * 4].view(torch.float32)
    on = buf[end - 256:end - 256 + row].view(torch.bfloat16).view(n, h, hd)
    before = buf[:end].clone()
    for call, ins in ((fm.paged_cross_attention, args), (fm.paged_gqa_decode_shared, shared)):
        want = call(*ins)
        got = call(*ins, out=beside[0], lse=beside[1].view(n, h))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for over in (dict(out=on), dict(lse=buf[256:256 + n * h * 4].view(torch.float32).view(n, h))):
            with pytest.raises((fm.FP8MLAError, ValueError)):
                call(*ins, **over)
    assert torch.equal(buf[:end], before) and fm.last_device_error() == 0
