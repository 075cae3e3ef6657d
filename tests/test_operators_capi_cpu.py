"""Host-side refusals of the rotary, append, read-back and 4-bit decode entry points (nothing is launched)."""

import pytest

import paged_decode_attention_fp8_gb300 as fm

P = 1 << 20  # stands for a device pointer; never followed


def _table(**over):
    a = dict(f=P, half=32, n=100, factor=1.0, table=P)
    a.update(over)
    return fm.lib().rotary_table(a["f"], a["half"], a["n"], a["factor"], a["table"], None)


@pytest.mark.parametrize("over", [dict(half=0), dict(half=4097), dict(n=-1), dict(factor=0.0), dict(factor=-1.0),
                                  dict(factor=float("nan")), dict(factor=float("inf")), dict(f=None),
                                  dict(table=None), dict(f=P + 4), dict(table=P + 4), dict(n=1 << 60)])
def test_table_refusals(over):
    assert _table(**over) == 1


def test_empty_table():
    assert _table(n=0, f=None, table=None) == 0


def _apply(**over):
    a = dict(q=P, qs=(4096, 128), qo=P, qos=(4096, 128), h_q=32, k=P, ks=(1024, 128), ko=P, kos=(1024, 128), h_k=8,
             dtype=0, pos=P, wide=0, table=P, n_pos=64, n=4, hd=128, rot=128, off=0, inter=0, inv=0)
    a.update(over)
    return fm.lib().rotary_apply(a["q"], *a["qs"], a["qo"], *a["qos"], a["h_q"], a["k"], *a["ks"], a["ko"], *a["kos"],
                                 a["h_k"], a["dtype"], a["pos"], a["wide"], a["table"], a["n_pos"], a["n"], a["hd"],
                                 a["rot"], a["off"], a["inter"], a["inv"], None)


@pytest.mark.parametrize("over", [dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(h_q=0), dict(h_k=-1),
                                  dict(pos=None), dict(table=None), dict(table=P + 4), dict(n_pos=0), dict(n=-1),
                                  dict(hd=1), dict(hd=8194), dict(rot=0), dict(rot=7), dict(rot=130), dict(off=-2),
                                  dict(rot=64, off=66), dict(q=P + 1), dict(dtype=2, ko=P + 2)])
def test_apply_refusals(over):
    assert _apply(**over) == 1


def test_apply_unknown_type_and_no_tokens():
    assert _apply(dtype=3) == 2
    assert _apply(n=0, q=None, k=None, pos=None, table=None) == 0


def _append(**over):
    a = dict(k=P, ks=(1024, 128), v=P, vs=(1024, 128), slots=P, n=4, h_kv=8, hd=128, page=16, blocks=64,
             dtype=fm.KV_E2M1, kc=P, vc=P, k_scale=P, v_scale=P, k_rows=None, v_rows=None, k_blk=P, v_blk=P, pos=P,
             wide=0, table=P, n_pos=64, rot=128, off=0, inter=0, q=P, qs=(4096, 128), qo=P, h_q=32)
    a.update(over)
    return fm.lib().paged_kv_append(a["k"], *a["ks"], a["v"], *a["vs"], a["slots"], a["n"], a["h_kv"], a["hd"],
                                    a["page"], a["blocks"], a["dtype"], a["kc"], a["vc"], a["k_scale"], a["v_scale"],
                                    a["k_rows"], a["v_rows"], a["k_blk"], a["v_blk"], a["pos"], a["wide"], a["table"],
                                    a["n_pos"], a["rot"], a["off"], a["inter"], a["q"], *a["qs"], a["qo"], a["h_q"],
                                    None)


@pytest.mark.parametrize("over", [
    dict(k=None), dict(v=None), dict(vc=None), dict(kc=None), dict(slots=None), dict(n=-1), dict(h_kv=0), dict(hd=24),
    dict(hd=0), dict(hd=1040), dict(page=0), dict(blocks=0), dict(k_scale=None), dict(v_blk=None), dict(k_rows=P),
    dict(ks=(1020, 128)), dict(vs=(1024, 4)), dict(k=P + 8), dict(vc=P + 8), dict(pos=None), dict(table=P + 8),
    dict(n_pos=0), dict(rot=0), dict(rot=24), dict(rot=16), dict(rot=144), dict(off=8), dict(rot=64, off=8),
    dict(rot=64, off=72), dict(rot=64, off=-16), dict(inter=1, rot=64, off=8), dict(qo=None), dict(h_q=0),
    dict(q=P + 2), dict(qs=(4096, 4)), dict(table=None), dict(blocks=1 << 28),
    dict(n=1 << 28), dict(dtype=fm.KV_E4M3), dict(dtype=fm.KV_E4M3, k_blk=None, v_blk=None, k_rows=P),
    dict(dtype=fm.KV_E4M3, k_blk=None, v_blk=None, k_scale=None, k_rows=P),
    dict(dtype=fm.KV_E4M3, k_blk=None, v_blk=None, k_scale=None, v_scale=None, k_rows=P, v_rows=P + 2)])
def test_append_refusals(over):
    assert _append(**over) == 1


@pytest.mark.parametrize("code", [fm.KV_E4M3FNUZ, fm.KV_E5M2, fm.KV_OTHER, 5])
def test_append_read_foreign_encodings(code):
    assert _append(dtype=code) == 2
    assert _read(dtype=code) == 2


def test_append_no_tokens():
    assert _append(n=0, k=None, v=None, vc=None, v_scale=None, v_blk=None, q=None, slots=None, pos=None) == 0


def _read(**over):
    a = dict(cache=P, dtype=fm.KV_E2M1, scale=P, rows=None, blk=P, slots=P, n=4, h_kv=8, hd=128, page=16, blocks=64,
             out=P)
    a.update(over)
    return fm.lib().paged_cache_read(a["cache"], a["dtype"], a["scale"], a["rows"], a["blk"], a["slots"], a["n"],
                                     a["h_kv"], a["hd"], a["page"], a["blocks"], a["out"], None)


@pytest.mark.parametrize("over", [dict(cache=None), dict(scale=None), dict(blk=None), dict(rows=P), dict(slots=None),
                                  dict(out=None), dict(out=P + 8), dict(cache=P + 8), dict(hd=24), dict(hd=1040),
                                  dict(n=-1), dict(h_kv=0), dict(page=0), dict(blocks=0), dict(n=1 << 28),
                                  dict(blocks=1 << 28), dict(dtype=fm.KV_E4M3),
                                  dict(dtype=fm.KV_E4M3, blk=None, rows=P), dict(dtype=fm.KV_E4M3, blk=None, hd=12)])
def test_read_refusals(over):
    assert _read(**over) == 1


def test_read_nothing():
    assert _read(n=0, cache=None, slots=None, out=None) == 0


def _decode(**over):
    a = dict(q=P, kc=P, vc=P, kb=P, vb=P, blocks=64, ks=P, vs=P, bt=P, mb=8, sl=P, scale=0.08, q_len=1, mask=None,
             window=0, sinks=None, splits=1, ws=P, wsb=1 << 40, out=P, lse=P, bs=2, h_q=32, h_kv=8, hd=128, page=16)
    a.update(over)
    return fm.lib().paged_gqa_decode_fp4(a["q"], a["kc"], a["vc"], a["kb"], a["vb"], a["blocks"], a["ks"], a["vs"],
                                         a["bt"], a["mb"], a["sl"], a["scale"], a["q_len"], a["mask"], a["window"],
                                         a["sinks"], a["splits"], a["ws"], a["wsb"], a["out"], a["lse"], a["bs"],
                                         a["h_q"], a["h_kv"], a["hd"], a["page"], None)


@pytest.mark.parametrize("over", [dict(hd=96), dict(hd=512), dict(page=8), dict(page=48), dict(page=512), dict(h_q=30),
                                  dict(h_q=0), dict(h_kv=0), dict(q_len=0), dict(q_len=17), dict(q_len=16, h_q=72),
                                  dict(window=-1), dict(splits=-1), dict(scale=0.0), dict(scale=float("nan")),
                                  dict(blocks=0), dict(mb=0), dict(bs=-1), dict(q=None), dict(kc=None), dict(vb=None),
                                  dict(ks=None), dict(bt=None), dict(sl=None), dict(out=None), dict(lse=None),
                                  dict(q=P + 8), dict(kc=P + 8), dict(vb=P + 4), dict(out=P + 2),
                                  dict(splits=2, mb=64, ws=None), dict(splits=2, mb=64, ws=P + 64),
                                  dict(splits=0, mb=4096, ws=None), dict(blocks=1 << 27), dict(mb=1 << 28)])
def test_decode_refusals(over):
    assert _decode(**over) == 1


def test_decode_workspace_and_empty_batch():
    assert _decode(splits=2, mb=64, wsb=256) == 3
    assert _decode(bs=0, q=None, out=None, lse=None) == 0


def test_workspace_of_each_layout():
    size = fm.gqa_fp4_workspace_bytes
    slot = 8 * 128 * 4 + 8 * 8  # eight columns of 128 floats and a pair of floats each
    assert size(3, 8, 2, 128, 4096, num_splits=1) == 0
    # short contexts: one CTA or one cluster each, longer ones where those come to fill the GPU (152 SMs here)
    assert size(3, 8, 2, 128, 2688) == 0 < size(3, 8, 2, 128, 2704)
    assert size(30, 8, 2, 128, 6144) == 0 < size(30, 8, 2, 128, 6160)
    assert size(50, 8, 2, 128, 2016) == 0 < size(50, 8, 2, 128, 2032)
    assert size(100, 8, 2, 128, 1536) == 0 < size(100, 8, 2, 128, 1552)
    assert size(2000, 8, 2, 128, 8192) == 0                 # more sequences than a CTA sums
    assert size(3, 8, 2, 128, 4096, num_splits=4) == 24 * slot
    # at most one shard per 128 keys, however many are asked for; a window bounds the keys
    assert size(1, 4, 1, 128, 1000, num_splits=100) == 8 * 8 * 128 * 4 + 8 * 8 * 8
    assert size(1, 4, 1, 128, 16, num_splits=100) == 0
    assert size(1, 4, 1, 128, 100000, window=100, num_splits=100) == 0
    # sixteen columns a tile past eight
    assert size(1, 24, 2, 64, 256, num_splits=2) == 4 * 16 * 64 * 4 + 4 * 16 * 8
    auto = size(1, 4, 1, 128, 1 << 17)                      # two states a piece, and the line of tiles
    assert auto >= 2 * slot and auto % 256 == 0
    for bad in (dict(head_dim=96), dict(h_q=5), dict(q_len=17), dict(window=-1), dict(num_splits=-1), dict(bs=0)):
        a = dict(bs=1, h_q=4, h_kv=2, head_dim=128, max_seqlen=1 << 17)
        a.update(bad)
        assert size(**a) == 0


def test_the_other_entries_refuse_the_4_bit_encoding():
    lib = fm.lib()
    assert lib.fp8_paged_cache_write(P, 1024, P, 4, 8, 128, 16, 64, fm.KV_E2M1, P, None, P, None) == 2
    assert lib.paged_gqa_decode(P, P, P, fm.KV_E2M1, 64, P, P, P, 8, P, 0.08, 1, P, 1 << 40, P, P, 2, 32, 8, 128, 16,
                                None) == 2
