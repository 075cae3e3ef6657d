"""Host-side refusals of cross attention, shared prefixes and the merge (nothing is launched, no GPU needed)."""

import ctypes

import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm

P = 1 << 40  # stand for device pointers; never followed
OUT, LSE, WS = P + (1 << 32), P + (2 << 32), P + (3 << 32)


def _cross(**over):
    a = dict(q=P, qs=(4096, 128), kc=P, vc=P, dtype=fm.KV_E4M3, blocks=64, ks=P, vs=P, rows=0, starts=P, bt=P, mb=8, kl=P,
             scale=0.08, ws=WS, wsb=1 << 40, out=OUT, os=(4096, 128), lse=LSE, fo=0, fl=0, n=10, bs=2, h_q=32, h_kv=8,
             hd=128, page=16)
    a.update(over)
    return fm.lib().paged_cross_attention(
        a["q"], *a["qs"], a["kc"], a["vc"], a["dtype"], a["blocks"], a["ks"], a["vs"], a["rows"], a["starts"], a["bt"],
        a["mb"], a["kl"], a["scale"], a["ws"], a["wsb"], a["out"], *a["os"], a["lse"], a["fo"], a["fl"], a["n"], a["bs"],
        a["h_q"], a["h_kv"], a["hd"], a["page"], None)


CROSS_BAD = [
    dict(q=None), dict(kc=None), dict(vc=None), dict(ks=None), dict(vs=None), dict(bt=None), dict(kl=None), dict(out=None),
    dict(lse=None), dict(ws=None), dict(ws=WS + 64), dict(q=P + 8), dict(kc=P + 8), dict(vc=P + 4), dict(out=OUT + 2),
    dict(lse=LSE + 2), dict(ks=P + 2), dict(vs=P + 8, rows=1), dict(starts=P + 1), dict(bt=P + 2), dict(kl=P + 3),
    dict(qs=(4096, 124)), dict(qs=(4090, 128)), dict(os=(4096, 4)), dict(hd=96), dict(hd=256), dict(page=8), dict(page=48),
    dict(page=512), dict(h_q=30), dict(h_q=0), dict(h_kv=0), dict(blocks=0), dict(mb=0), dict(n=-1), dict(bs=-1),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(starts=None, n=1), dict(mb=1 << 27),
    dict(blocks=1 << 24), dict(n=1 << 26),
    # outputs that share memory with each other, with themselves, with the queries (otherwise than in their place)
    dict(out=P, os=(4096, 256)), dict(out=P + 256), dict(lse=P), dict(lse=OUT), dict(ws=OUT), dict(ws=LSE), dict(ws=P),
    dict(os=(0, 128)), dict(os=(4096, 64))]


@pytest.mark.parametrize("over", CROSS_BAD)
def test_cross_refusals(over):
    assert _cross(**over) == 1


def _shared(**over):
    a = dict(q=P, kc=P, vc=P, dtype=fm.KV_E4M3, blocks=64, ks=P, vs=P, rows=0, pt=P, pb=4, pl=P, ps=P, np=2, bt=P, mb=8,
             sl=P, scale=0.08, q_len=1, mask=None, sinks=None, ws=WS, wsb=1 << 40, out=OUT, lse=LSE, bs=2, h_q=32, h_kv=8,
             hd=128, page=16)
    a.update(over)
    return fm.lib().paged_gqa_decode_shared(
        a["q"], a["kc"], a["vc"], a["dtype"], a["blocks"], a["ks"], a["vs"], a["rows"], a["pt"], a["pb"], a["pl"], a["ps"],
        a["np"], a["bt"], a["mb"], a["sl"], a["scale"], a["q_len"], a["mask"], a["sinks"], a["ws"], a["wsb"], a["out"],
        a["lse"], a["bs"], a["h_q"], a["h_kv"], a["hd"], a["page"], None)


@pytest.mark.parametrize("over", [
    dict(q=None), dict(kc=None), dict(pt=None), dict(pl=None), dict(ps=None), dict(bt=None), dict(sl=None), dict(out=None),
    dict(lse=None), dict(ws=None), dict(ws=WS + 16), dict(q=P + 2), dict(vc=P + 8), dict(pt=P + 2), dict(pl=P + 1),
    dict(ps=P + 2), dict(sinks=P + 2), dict(sl=P + 2), dict(ks=P + 4, rows=1), dict(q_len=0), dict(q_len=33), dict(np=-1),
    dict(pb=0), dict(mb=0), dict(bs=-1), dict(hd=80), dict(page=24), dict(h_q=12), dict(scale=0.0), dict(blocks=0),
    dict(blocks=1 << 24), dict(pb=1 << 27), dict(out=P + 128), dict(lse=OUT), dict(ws=OUT)])
def test_shared_refusals(over):
    assert _shared(**over) == 1


@pytest.mark.parametrize("call", [_cross, _shared])
def test_foreign_encodings_small_workspaces_and_nothing_to_do(call):
    for code in (fm.KV_E4M3FNUZ, fm.KV_E5M2, fm.KV_E2M1, fm.KV_OTHER):
        assert call(dtype=code) == 2
    assert call(wsb=64) == 3
    assert call(bs=0, **(dict(n=0) if call is _cross else {}), q=None, out=None, lse=None, bt=None) == 0


def test_workspace_sizes():
    small, large = fm.cross_workspace_bytes(1, 1, 8, 2, 64, 128), fm.cross_workspace_bytes(4096, 4, 32, 8, 128, 1 << 15)
    assert 0 < small < large and small % 256 == 0
    # at most two pieces of 256 rows a share, one share an SM (152 where none is asked)
    assert large < 2 * 160 * 256 * (128 * 4 + 8) + (1 << 16)
    assert fm.cross_workspace_bytes(1 << 20, 1, 64, 8, 128, 1 << 20) < 2 * large  # it does not grow with the batch
    for bad in ((-1, 1, 8, 2, 64, 128), (1, -1, 8, 2, 64, 128), (1, 1, 7, 2, 64, 128), (1, 1, 8, 2, 96, 128),
                (1, 1, 8, 2, 64, -1), (1 << 28, 1, 8, 2, 64, 128)):
        assert fm.cross_workspace_bytes(*bad) == 0
    one = fm.gqa_shared_workspace_bytes(64, 1, 32, 8, 128, 1, 1 << 15, 1024)
    assert one >= 2 * 64 * 32 * (128 * 4 + 8)  # both halves' sums
    for bad in ((64, 0, 32, 8, 128, 1, 64, 64), (64, 33, 32, 8, 128, 1, 64, 64), (64, 1, 32, 8, 128, -1, 64, 64)):
        assert fm.gqa_shared_workspace_bytes(*bad) == 0


def _merge(parts=2, outs=None, strides=(4096, 128), lses=None, out=OUT, to=(4096, 128), lse=LSE, n=4, heads=32, dim=128):
    ptr = (ctypes.c_void_p * 9)(*(outs or [P + i * (1 << 24) for i in range(9)]))
    sums = (ctypes.c_void_p * 9)(*(lses or [P + (1 << 30) + i * (1 << 20) for i in range(9)]))
    tokens, heads_ = ((ctypes.c_int64 * 9)(*([s] * 9)) for s in strides)
    return fm.lib().attention_merge(ptr, tokens, heads_, sums, parts, out, *to, lse, n, heads, dim, None)


@pytest.mark.parametrize("over", [
    dict(parts=0), dict(parts=9), dict(n=-1), dict(heads=0), dict(dim=0), dict(dim=12), dict(dim=1032), dict(out=None),
    dict(lse=None), dict(out=OUT + 8), dict(lse=LSE + 2), dict(strides=(4096, 4)), dict(to=(4100, 128)), dict(to=(0, 128)),
    dict(outs=[P, None] + [P] * 7), dict(outs=[P, P + 8] + [P] * 7), dict(lses=[P, None] + [P] * 7),
    dict(lses=[P, P + 2] + [P] * 7), dict(out=P + 256), dict(lse=P), dict(lse=OUT), dict(lse=P + (1 << 30)),
    dict(out=P + (1 << 30)), dict(n=1 << 26)])
def test_merge_refusals(over):
    assert _merge(**over) == 1


def test_merge_of_nothing():
    assert _merge(n=0, out=None, lse=None) == 0


X = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
CACHE, ONE, LENS = torch.zeros((2, 2, 16, 64), dtype=torch.uint8), torch.ones(1), torch.zeros(4, dtype=torch.int32)
TABLE = torch.zeros((4, 1), dtype=torch.int32)


def _py_cross(q=X, k_scale=ONE, v_scale=ONE, **kw):
    fm.paged_cross_attention(q, CACHE, CACHE, TABLE, LENS, k_scale, v_scale, **kw)


def _py_shared(q=X, k_scale=ONE, v_scale=ONE, **kw):
    fm.paged_gqa_decode_shared(q, CACHE, CACHE, TABLE[:1], LENS[:1], LENS[:2], TABLE, LENS, k_scale, v_scale, **kw)


def _py_merge(outs=X, lses=X[..., 0].float(), **kw):
    fm.attention_merge([X, outs], [X[..., 0].float(), lses], **kw)


@pytest.mark.parametrize("call,name", [(_py_cross, n) for n in ("q", "k_scale", "v_scale", "out", "lse")] +
                         [(_py_shared, n) for n in ("q", "k_scale", "v_scale", "sinks", "out", "lse")] +
                         [(_py_merge, n) for n in ("out", "lse")])
def test_a_gradient_that_would_be_lost_is_refused(call, name):
    t = (X if name in ("q", "out") else ONE).clone().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        call(**{name: t})
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # the next refusal: these are on the CPU
        call(**{name: t})


def test_merge_takes_lists_of_the_same_length():
    with pytest.raises(ValueError, match="parts"):
        fm.attention_merge([X] * 2, [X[..., 0].float()])
    with pytest.raises(ValueError, match="parts"):
        fm.attention_merge([], [])
    with pytest.raises(ValueError, match="parts"):
        fm.attention_merge([X] * 9, [X] * 9)
    with pytest.raises(ValueError, match="lists"):
        fm.attention_merge(X, X)
    with pytest.raises(ValueError, match="CUDA"):
        fm.attention_merge([X] * 2, [X[..., 0].float()] * 2)
