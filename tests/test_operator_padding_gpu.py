"""Rows of padding: zeros in outputs that a call makes, left alone in those it is given."""

import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
NAN = float("nan")


def _soiled(*shapes):
    """Memory of these sizes, full of NaN, is what the next allocations get."""
    for shape, dtype in shapes:
        torch.full(shape, NAN, dtype=dtype, device=DEV)


def _inputs(n, heads, hd, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((n, heads, hd), generator=g).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("hq,hk,hd,rot,offset,interleaved", [
    (32, 8, 128, 128, 0, False), (5, 1, 96, 64, 32, True), (3, 2, 80, 16, 8, False), (4, 0, 62, 30, 7, False),
    (1, 1, 600, 600, 0, True), (40, 8, 192, 64, 128, True)])
def test_new_outputs_of_the_rotation(dtype, hq, hk, hd, rot, offset, interleaved):
    n = 13
    q, k = _inputs(n, hq, hd, dtype, 1), _inputs(n, hk, hd, dtype, 2) if hk else None
    f, _ = fm.rotary_frequencies(rot)
    table = fm.rotary_table(f, 50)
    pos = torch.tensor([0, -1, 49, 3, 50, -7, 1 << 40, 5, 6, 7, -1, 9, -(1 << 40)], device=DEV)
    pad = (pos < 0) | (pos >= 50)
    kw = dict(interleaved=interleaved, rot_offset=offset)
    given = [torch.full_like(t, -7.0) if t is not None else None for t in (q, k)]
    want = fm.rotary_apply(q, k, pos, table, q_out=given[0], k_out=given[1], **kw)
    assert fm.last_device_error() == fm.DEV_BAD_POSITION
    for t in want:
        assert t is None or bool((t[pad] == -7.0).all())
    _soiled(*[(t.shape, dtype) for t in (q, k) if t is not None])
    for got, w in zip(fm.rotary_apply(q, k, pos, table, **kw), want):
        if w is not None:
            assert bool((got[pad] == 0).all()) and torch.equal(got[~pad], w[~pad])
    if k is not None:  # one given, one made
        out = torch.full_like(k, -7.0)
        _soiled((q.shape, dtype))
        made, _ = fm.rotary_apply(q, k, pos, table, k_out=out, **kw)
        assert bool((made[pad] == 0).all()) and bool((out[pad] == -7.0).all()) and torch.equal(out[~pad], want[1][~pad])
        out = torch.full_like(q, -7.0)
        _soiled((k.shape, dtype))
        _, made = fm.rotary_apply(q, k, pos, table, q_out=out, **kw)
        assert bool((made[pad] == 0).all()) and bool((out[pad] == -7.0).all())
    assert fm.last_device_error() == fm.DEV_BAD_POSITION


@pytest.mark.parametrize("hd,h_q", [(64, 4), (128, 32), (192, 3), (576, 16), (1024, 2), (16, 1)])
@pytest.mark.parametrize("kind", ["tensor", "fp4"])
def test_new_queries_of_the_append(hd, h_q, kind):
    if kind == "fp4" and hd == 16:
        pytest.skip("no half layout of 4 bits so narrow")
    n = 11
    x = _inputs(n, h_q + 2, hd, torch.bfloat16, 3)
    f, _ = fm.rotary_frequencies(min(hd, 64))
    table, slots = fm.rotary_table(f, 50), torch.arange(n, dtype=torch.int32, device=DEV)
    slots[3] = -1  # skips K and V, not the queries
    pos = torch.tensor([0, -1, 49, 3, 50, -7, 1, 2, -1, 9, 10], dtype=torch.int32, device=DEV)
    pad = (pos < 0) | (pos >= 50)
    one = torch.tensor([0.01], device=DEV)

    def call(**kw):
        wide = hd // 2 if kind == "fp4" else hd
        c = [torch.zeros((1, 1, 16, wide), dtype=torch.uint8, device=DEV) for _ in range(2)]
        if kind == "fp4":
            kw.update({s + "_block_scales": torch.zeros((1, 1, 16, hd // 16), dtype=torch.uint8, device=DEV)
                       for s in "kv"})
        q = fm.paged_kv_append(x[:, h_q:h_q + 1], x[:, h_q + 1:], slots, *c, positions=pos, table=table, k_scale=one,
                               v_scale=one, q=x[:, :h_q], **kw)
        return [q] + c + [kw[s + "_block_scales"] for s in "kv" if kind == "fp4"]

    want = call(q_out=torch.full((n, h_q, hd), -7.0, dtype=torch.bfloat16, device=DEV))
    assert bool((want[0][pad] == -7.0).all())
    _soiled(((n, h_q, hd), torch.bfloat16))
    got = call()
    assert bool((got[0][pad] == 0).all()) and torch.equal(got[0][~pad], want[0][~pad])
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    assert fm.last_device_error() == fm.DEV_BAD_POSITION
