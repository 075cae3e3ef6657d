"""Merges of parts whose LSE is +inf: no weight is defined, so the row is NaN and stays visible in later merges."""

import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
INF = float("inf")


@pytest.mark.parametrize("parts", [1, 2, 3, 8])
@pytest.mark.parametrize("others", [0.5, -INF, INF, float("nan")])
def test_an_infinite_part(parts, others):
    outs = [torch.randn((5, 3, 64), device=DEV).to(torch.bfloat16) for _ in range(parts)]
    lses = [torch.randn((5, 3), device=DEV) for _ in range(parts)]
    clean = fm.attention_merge(outs, lses)
    for l in lses:
        l[2, 1] = others
    lses[parts // 2][2, 1] = INF
    out, lse = fm.attention_merge(outs, lses)
    assert bool(out[2, 1].isnan().all()) and bool(lse[2, 1].isnan())
    assert int(lse.isnan().sum()) == 1 and int(out.isnan().sum()) == 64
    rest = torch.ones((5, 3), dtype=torch.bool, device=DEV)
    rest[2, 1] = False
    assert torch.equal(out[rest], clean[0][rest]) and torch.equal(lse[rest], clean[1][rest])
    # with another part, which does not bring it back to a number
    again = fm.attention_merge([out, outs[0]], [lse, torch.zeros_like(lse)])
    assert bool(again[0][2, 1].isnan().all()) and bool(again[1][2, 1].isnan()) and int(again[1].isnan().sum()) == 1
