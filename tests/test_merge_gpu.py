"""The merge of partial results on the GPU against the float64 oracle.

Tolerances, before any run: weights from the approximate 2^x, sums and products in float32 are off by 2^-18 at most of
sum w |out| (2^-21 of the exponent's rounding at |lse| <= 64 times log2 e, 2^-22 of 2^x, a few 2^-24), then the rounding
to bf16, 2^-8 of the value; the LSE by 2^-20 and 2^-22 of its size.
"""

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from oracle import ragged

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _parts(seed, parts, n, heads, dim, empty=0.2):
    g = torch.Generator().manual_seed(seed)
    outs = [torch.randn((n, heads, dim), generator=g).to(torch.bfloat16) for _ in range(parts)]
    lses = [torch.randn((n, heads), generator=g) * 8 for _ in range(parts)]
    for o, l in zip(outs, lses):
        none = torch.rand((n, heads), generator=g) < empty
        none[-1] = n > 1  # a token that no part has a key for
        o[none], l[none] = float("nan"), -float("inf")  # whatever such a row holds
    return outs, lses


def _check(got, outs, lses):
    out, lse = (x.double().cpu().numpy() for x in got)
    want = ragged.merge(outs, lses)
    size = ragged.merge([o.abs() for o in outs], lses)[0]
    assert np.array_equal(lse == -np.inf, want[1] == -np.inf)
    assert np.all(np.abs(out - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -18 * size)
    finite = np.isfinite(want[1])
    assert np.all(np.abs(lse[finite] - want[1][finite]) <= 2.0 ** -20 + 2.0 ** -22 * np.abs(want[1][finite]))


@pytest.mark.parametrize("parts", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("n,heads,dim", [(1, 1, 8), (3, 5, 64), (130, 32, 128), (17, 16, 512), (2, 3, 1024), (9, 7, 72)])
def test_shapes(parts, n, heads, dim):
    outs, lses = _parts(parts, parts, n, heads, dim)
    got = fm.attention_merge([o.to(DEV) for o in outs], tuple(l.to(DEV) for l in lses))
    _check(got, outs, lses)


def test_strides_and_in_place():
    outs, lses = _parts(1, 3, 20, 4, 64)
    dev = [torch.empty((20, 5, 80), dtype=torch.bfloat16, device=DEV)[:, :4, 8:72].copy_(outs[0]),
           torch.empty((4, 20, 64), dtype=torch.bfloat16, device=DEV).transpose(0, 1).copy_(outs[1]),
           torch.empty((20, 4, 64), dtype=torch.bfloat16, device=DEV).copy_(outs[2])]
    l = [x.to(DEV) for x in lses]
    want = fm.attention_merge(dev, l)
    _check(want, outs, lses)
    for i in range(3):
        again = [x.clone(memory_format=torch.preserve_format) if j != i else x for j, x in enumerate(dev)]
        keep = dev[i].clone()
        got, _ = fm.attention_merge(again, l, out=again[i])
        assert got is again[i] and torch.equal(got, want[0])
        dev[i].copy_(keep)


def test_a_nan_lse_and_far_ones():
    outs, lses = _parts(2, 2, 6, 2, 64, empty=0.0)
    lses[0][0, 0], lses[1][1, 1] = float("nan"), 3e38
    lses[0][2], lses[1][2] = -3e38, -3e38
    out, lse = fm.attention_merge([o.to(DEV) for o in outs], [l.to(DEV) for l in lses])
    assert bool(out[0, 0].isnan().all()) and bool(lse[0, 0].isnan()) and int(lse.isnan().sum()) == 1
    assert torch.equal(out[1, 1].cpu(), outs[1][1, 1])
    mean = (outs[0][2].double() + outs[1][2].double()) / 2
    assert bool(((out[2].cpu().double() - mean).abs() <= 2.0 ** -8 * mean.abs() + 1e-6).all())


def test_nothing():
    out, lse = fm.attention_merge([torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)] * 2,
                                  [torch.empty((0, 4), device=DEV)] * 2)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
