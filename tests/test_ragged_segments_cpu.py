"""Batches of more sequences and prefixes than the device counts through (nothing is launched)."""

import pytest

import paged_decode_attention_fp8_gb300 as fm
from tests.test_ragged_capi_cpu import P, _cross, _shared

MOST = 1 << 26
FAR = dict(out=P + (1 << 44), lse=P + (1 << 45), ws=P + (1 << 46))  # clear of the inputs


@pytest.mark.parametrize("call,over", [
    (_cross, dict(bs=MOST + 1)), (_cross, dict(bs=(1 << 31) - 1)), (_cross, dict(bs=MOST + 1, n=MOST + 1, h_q=8)),
    (_shared, dict(bs=MOST, np=1, h_q=8)), (_shared, dict(bs=1, np=MOST)), (_shared, dict(np=(1 << 31) - 1))])
def test_too_many(call, over):
    assert call(**over, **FAR, wsb=64) == 1


def test_most():
    assert _cross(bs=MOST, **FAR, wsb=64) == 3  # the next refusal: the workspace
    assert _shared(bs=MOST - 2, h_q=8, **FAR, wsb=64) == 3
    assert fm.cross_workspace_bytes(10, MOST, 8, 8, 64, 128) > 0 == fm.cross_workspace_bytes(10, MOST + 1, 8, 8, 64, 128)
    assert fm.gqa_shared_workspace_bytes(1, 1, 8, 8, 64, MOST - 1, 128, 128) > 0
    assert fm.gqa_shared_workspace_bytes(1, 1, 8, 8, 64, MOST, 128, 128) == 0
