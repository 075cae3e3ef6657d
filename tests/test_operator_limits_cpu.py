"""Size limits and alignments of the rotary, append, read-back and 4-bit decode entries (nothing is launched: what
passes the limits is stopped by a later check, or has no token)."""

import pytest

from tests.test_operators_capi_cpu import P, _append, _apply, _decode, _read


@pytest.mark.parametrize("h_kv,page", [(1, 256), (1, 16), (2, 256), (8, 64)])
def test_decode_takes_fewer_than_2_to_32_rows(h_kv, page):
    most = (1 << 32) // (h_kv * page)
    a = dict(h_kv=h_kv, h_q=4 * h_kv, page=page, splits=2, mb=1024 // page, wsb=256)
    assert _decode(**a, blocks=most - 1) == 3  # the workspace is too small: past every other check of sizes
    assert _decode(**a, blocks=most) == 1


@pytest.mark.parametrize("page", [16, 64, 256])
def test_slots_are_below_2_to_31(page):
    most = (1 << 31) // page
    for call in (_append, _read):
        assert call(n=0, h_kv=1, page=page, blocks=most - 1) == 0
        assert call(n=0, h_kv=1, page=page, blocks=most) == 1


def test_rows_of_a_call_are_below_2_to_31():
    assert _append(n=(1 << 31) // 8, h_kv=8, h_q=1) == 1 and _append(n=(1 << 31) // 32, h_kv=1, h_q=32) == 1
    assert _read(n=(1 << 31) // 8, h_kv=8) == 1


@pytest.mark.parametrize("call,over", [
    (_apply, dict(pos=P + 2)), (_apply, dict(pos=P + 4, wide=1)),
    (_append, dict(slots=P + 2)), (_append, dict(pos=P + 1)), (_append, dict(pos=P + 4, wide=1)),
    (_read, dict(slots=P + 2)), (_decode, dict(ks=P + 2)), (_decode, dict(vs=P + 1)), (_decode, dict(bt=P + 2)),
    (_decode, dict(sl=P + 3)), (_decode, dict(sinks=P + 2)), (_decode, dict(lse=9 * P + 2))])
def test_misaligned_indexes_and_scales_are_refused(call, over):
    """Other arguments as in a call that is not refused for another reason."""
    apart = {_apply: dict(qo=2 * P, k=3 * P, ko=4 * P),
             _append: dict(v=2 * P, kc=3 * P, vc=4 * P, k_blk=5 * P, v_blk=6 * P, q=7 * P, qo=8 * P),
             _read: dict(cache=2 * P, blk=3 * P, out=4 * P), _decode: dict(q=2 * P, out=3 * P, lse=4 * P)}[call]
    assert call(**{**apart, **over}) == 1


def test_unknown_layout_bits_are_refused():
    assert _apply(inter=8) == 1 and _apply(inter=-1) == 1 and _append(n=0, inter=4) == 1 and _append(n=0, inter=-1) == 1
    assert _apply(n=0, inter=7) == 0 and _append(n=0, inter=3) == 0
