"""GQA and dense MLA decode with row scales far below one: rows of 0, of the smallest floats and of 2^-115.

A V scale below 2^-110 counts as 2^-110: beside ordinary rows that is nothing (2^-101 of a weight), so the tolerances of
the tests with ordinary scales apply; where a whole sequence has such scales, the LSE holds and the output is below 2^-101.
"""

import numpy as np
import pytest
import torch

import oracle
import paged_decode_attention_fp8_gb300 as fm
from paged_decode_attention_fp8_gb300 import synthetic as syn
from tests.parity import assert_close, compare

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
FACTORS = [0.0, 2.0 ** -145, 2.0 ** -133, 2.0 ** -115, 2.0 ** -80]


def _scale_some(rng, s, part):
    """`part` of the rows times one of FACTORS each."""
    f = np.where(rng.random(s.shape) < part, rng.choice(FACTORS, s.shape), 1.0)
    return torch.from_numpy((s.double().numpy() * f).astype(np.float32))


@pytest.mark.parametrize("group", [4, 8])
@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("part", [0.01, 0.5])
def test_gqa_some_rows(group, splits, part):
    inp = syn.gqa_inputs(71, 3, [300, 40, 2000], h_q=2 * group, h_kv=2, spare_blocks=6)
    shape = tuple(inp.k_cache.shape[:3])
    ks = syn.per_row_scales(71, 50, shape, inp.k_scale)
    vs = _scale_some(np.random.default_rng(71), syn.per_row_scales(71, 51, shape, inp.v_scale), part)
    out, lse = fm.paged_gqa_decode_ext(inp.q.unsqueeze(1).to(DEV), inp.k_cache.to(DEV), inp.v_cache.to(DEV),
                                       inp.block_table.to(DEV), inp.seqlens.to(DEV), ks.to(DEV), vs.to(DEV),
                                       inp.softmax_scale, num_splits=splits)
    ro, rl = oracle.gqa_decode(inp.q, inp.k_cache, inp.v_cache, inp.block_table, inp.seqlens, ks.numpy(), vs.numpy(),
                               inp.softmax_scale)
    assert_close(compare(out[:, 0], lse[:, 0], ro, rl, "bf16"), "bf16")
    assert fm.last_device_error() == 0


@pytest.mark.parametrize("factor", FACTORS)
def test_gqa_all_rows(factor):
    inp = syn.gqa_inputs(72, 2, [300, 2000], h_q=8, h_kv=2, spare_blocks=6)
    shape = tuple(inp.k_cache.shape[:3])
    ks = syn.per_row_scales(72, 50, shape, inp.k_scale)
    vs = (syn.per_row_scales(72, 51, shape, inp.v_scale).double() * factor).float()
    out, lse = fm.paged_gqa_decode_ext(inp.q.unsqueeze(1).to(DEV), inp.k_cache.to(DEV), inp.v_cache.to(DEV),
                                       inp.block_table.to(DEV), inp.seqlens.to(DEV), ks.to(DEV), vs.to(DEV),
                                       inp.softmax_scale)
    ro, rl = oracle.gqa_decode(inp.q, inp.k_cache, inp.v_cache, inp.block_table, inp.seqlens, ks.numpy(), vs.numpy(),
                              inp.softmax_scale)
    if factor >= 2.0 ** -100:  # (brought back to an ordinary size, exactly)
        assert_close(compare(out[:, 0].double() / factor, lse[:, 0], ro / factor, rl, "bf16"), "bf16")
    assert float(out.abs().max()) <= 448 * max(2.0 ** -110, float(vs.max()))
    assert np.abs(lse[:, 0].double().cpu().numpy() - rl).max() <= 2e-3  # tests/parity.py


@pytest.mark.parametrize("part", [0.01, 0.5, 1.0])
@pytest.mark.parametrize("force_splits", [0, 3])
def test_mla(part, force_splits):
    inp, rows = syn.mla_row_scaled_inputs(73, 3, 2, 64, [700, 65, 2048], causal=True, spare_pages=3)
    small = _scale_some(np.random.default_rng(73), rows, part)
    sl = inp.seqlens.to(DEV)
    ts, ns = fm.get_metadata(sl, inp.h_q, inp.s_q, force_splits=force_splits)
    out, lse = fm.decode(inp.q.to(DEV), inp.kv_cache.to(DEV), inp.block_table.to(DEV), sl, small.to(DEV),
                         inp.softmax_scale, inp.causal, ts, ns, dot_mode="fp8")
    ro, rl = oracle.mla_decode(inp.q, inp.kv_cache, inp.block_table, inp.seqlens, small.numpy(), inp.softmax_scale,
                               inp.causal)
    if part < 1.0:
        assert_close(compare(out, lse, ro, rl, "fp8"), "fp8")
    else:
        assert float(out.abs().max()) <= 448 * max(2.0 ** -110, float(small.max()))
        live = np.isfinite(rl)
        assert np.abs(lse.double().cpu().numpy()[live] - rl[live]).max() <= 2e-3
    assert fm.last_device_error() == 0
