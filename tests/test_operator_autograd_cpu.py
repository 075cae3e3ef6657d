"""The rotary, append, read-back and 4-bit decode calls record nothing for autograd, and say so (no GPU needed)."""

import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm

X = torch.zeros((4, 2, 32), dtype=torch.bfloat16)
POS, TABLE = torch.zeros(4, dtype=torch.int32), torch.zeros((8, 16, 2))
CACHE, S8, ONE = torch.zeros((2, 2, 16, 32), dtype=torch.uint8), torch.zeros((2, 2, 16, 4)), torch.ones(1)


def _grad(t):
    return t.detach().clone().requires_grad_()


def _rotary(q=X, k=X, table=TABLE, **kw):
    fm.rotary_apply(q, k, POS, table, **kw)


def _append(k=X, v=X, k_scale=ONE, **kw):
    fm.paged_kv_append(k, v, POS, CACHE, CACHE.clone(), positions=POS, k_scale=k_scale, v_scale=ONE,
                       **{"table": TABLE, **kw})


def _read(scale=ONE, **kw):
    fm.paged_cache_read(CACHE, POS, scale=scale, **kw)


def _attend(q=X, k_scale=ONE, v_scale=ONE, **kw):
    fm.paged_gqa_decode_fp4(q, CACHE, CACHE, S8, S8, POS.view(4, 1), POS, k_scale, v_scale, **kw)


CALLS = [(_rotary, ("q", "k", "table", "q_out", "k_out")), (_append, ("k", "v", "k_scale", "q", "q_out", "table")),
         (_read, ("scale", "row_scales", "out")), (_attend, ("q", "k_scale", "v_scale", "sinks", "out", "lse"))]


@pytest.mark.parametrize("call,name", [(c, n) for c, names in CALLS for n in names])
def test_a_gradient_that_would_be_lost_is_refused(call, name):
    t = _grad(ONE if "scale" in name or name in ("sinks", "lse") else (TABLE if name == "table" else X))
    with pytest.raises(ValueError, match="gradient"):
        call(**{name: t})
    for off in (torch.no_grad, torch.inference_mode):
        with off(), pytest.raises(ValueError, match="CUDA"):  # the next refusal: these are on the CPU
            call(**{name: t})


def test_the_table_has_no_gradient_either():
    f, _ = fm.rotary_frequencies(32)
    with pytest.raises(ValueError, match="gradient"):
        fm.rotary_table(_grad(f), 4)
