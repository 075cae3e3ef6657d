"""The native marshalling loads without a GPU and refuses what it is not given on one."""

import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm


def test_calls_refuse_cpu_tensors_and_other_objects():
    x = torch.zeros((4, 2, 32), dtype=torch.bfloat16)
    pos, table = torch.zeros(4, dtype=torch.int32), torch.zeros((8, 16, 2))
    cache, scale = torch.zeros((2, 2, 16, 32), dtype=torch.uint8), torch.ones(1)
    s8 = torch.zeros((2, 2, 16, 4), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        fm.rotary_apply(x, None, pos, table)
    with pytest.raises(ValueError, match="q must be a tensor"):
        fm.rotary_apply(None, None, pos, table)
    with pytest.raises(ValueError, match="positions must be a tensor"):
        fm.rotary_apply(x, None, [0, 1, 2, 3], table)
    with pytest.raises(ValueError, match="CUDA"):
        fm.paged_kv_append(x, None, pos, cache, k_scale=scale)
    with pytest.raises(ValueError, match="CUDA"):
        fm.paged_cache_read(cache, pos, scale=scale)
    with pytest.raises(ValueError, match="CUDA"):
        fm.paged_gqa_decode_fp4(torch.zeros((1, 2, 64), dtype=torch.bfloat16), cache, cache, s8, s8,
                                torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32), scale, scale)


def test_a_missing_binding_raises(monkeypatch):
    monkeypatch.setattr(fm, "_binding", None)
    monkeypatch.setattr(fm.importlib, "import_module", lambda *a: (_ for _ in ()).throw(ImportError("none")))
    with pytest.raises(RuntimeError, match="binding"):
        fm._native()
