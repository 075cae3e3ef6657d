"""Q of cross attention as two E4M3 terms: exact from 2^-9.8 of a row's largest value on, else off by 2^-17.8 of it at most.

The largest value is scaled into (224, 448] and E4M3's last step is 2^-9: a first term and its rest are exact for bf16
values from 2^-2 on, which is 2^-9.8 of 224 at most, and off by 2^-10 else, 2^-17.8 of 224.  One key that has a one in
dim 1 and zeros elsewhere gives that value back as the LSE (2^-20 and 2^-21 of it for log2, 2^x and float32).
"""

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("tokens_each", [1, 100, 4096])
def test_small_values_of_a_row(hd, tokens_each):
    rng = np.random.default_rng(51)
    n = 4096
    largest = np.floor(rng.uniform(128, 256, n)) * 2.0 ** rng.integers(-3, 6, n)  # bf16: 8 bits
    x = np.floor(rng.uniform(128, 256, n)) / 128 * 2.0 ** np.floor(np.log2(largest) - rng.integers(1, 24, n))
    x *= rng.choice([-1, 1], n)
    q = torch.zeros((n, 1, hd), dtype=torch.float64)
    q[:, 0, 0], q[:, 0, 1] = torch.from_numpy(largest), torch.from_numpy(x)
    assert torch.equal(q.to(torch.bfloat16).double(), q)
    k = torch.zeros((1, 1, 16, hd), dtype=torch.uint8)
    k[0, 0, 0, 1] = 0x38
    k = k.to(DEV).view(torch.float8_e4m3fn)
    starts = torch.arange(0, n + tokens_each, tokens_each).clamp(max=n).to(torch.int32).to(DEV)
    bs, one = len(starts) - 1, torch.ones(1, device=DEV)
    _, lse = fm.paged_cross_attention(q.to(torch.bfloat16).to(DEV), k, k, torch.zeros((bs, 1), dtype=torch.int32, device=DEV),
                                      torch.ones(bs, dtype=torch.int32, device=DEV), one, one, softmax_scale=1.0,
                                      q_starts=starts)
    err = np.abs(lse[:, 0].double().cpu().numpy() - x)
    bound = np.where(np.abs(x) >= 2.0 ** -9.8 * largest, 0.0, largest * 2.0 ** -10 / 224)
    assert np.all(err <= bound + 2.0 ** -20 + 2.0 ** -21 * np.abs(x))
    assert fm.last_device_error() == 0
