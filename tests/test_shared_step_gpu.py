"""A decode step of samples of one prompt whose keys are rotated at their own positions: the prompt's from 0 on, the
samples' behind it."""

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from oracle.attention import as_bytes, e4m3_decode
from oracle.rotary import rotate
from tests import ragged_inputs as inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).to(DEV)


@pytest.mark.parametrize("hd", [64, 128])
def test_a_step_behind_a_prompt(hd):
    rng = np.random.default_rng(41)
    page, h_kv, h_q, prompt, own, unit = 16, 2, 8, 96, [5, 17, 1, 40], 0.02
    blocks = prompt // page + sum(-(-n // page) for n in own)
    caches = [torch.zeros((blocks, h_kv, page, hd), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    scale = torch.tensor([unit], device=DEV)
    f, factor = fm.rotary_frequencies(hd)
    table = fm.rotary_table(f, 256, factor=factor)
    perm = rng.permutation(blocks)
    ptable, at = perm[None, :prompt // page], prompt // page
    otable = np.zeros((4, 3), np.int64)
    for b, n in enumerate(own):
        c = -(-n // page)
        otable[b, :c] = perm[at:at + c]
        at += c
    rows = lambda n, h: torch.from_numpy(rng.standard_normal((n, h, hd))).to(torch.bfloat16)  # noqa: E731

    def append(pages, count, base, q=None):
        """Rows 0 .. count of these pages, at positions base on; (rotated keys, rotated queries)."""
        j = np.arange(count)
        k, v = rows(count, h_kv), rows(count, h_kv)
        slots = _i32(pages[j // page] * page + j % page)
        done = fm.paged_kv_append(k.to(DEV), v.to(DEV), slots, *caches, positions=_i32(j + base), table=table, k_scale=scale,
                                  v_scale=scale, q=None if q is None else q.to(DEV))
        want = rotate(k, j + base, f, factor=factor)
        for h in range(h_kv):  # what the cache holds: off by E4M3's half step, and the rotation in float32
            got = e4m3_decode(as_bytes(caches[0].cpu()))[pages[j // page], h, j % page] * unit
            assert np.all(np.abs(got - want[:, h]) <= 2.0 ** -4 * np.abs(want[:, h]) + 2.0 ** -10 * unit + 2.0 ** -20)
        return done

    append(ptable[0], prompt, 0)
    q = []
    for b, n in enumerate(own):
        x = rows(n, h_q)
        q.append(append(otable[b], n, prompt, x)[-1:])
        turned = rotate(x[-1:], np.array([prompt + n - 1]), f, factor=factor)[0]
        assert np.all(np.abs(q[-1][0].double().cpu().numpy() - turned) <= 2.0 ** -8 * np.abs(turned) + 2.0 ** -20)
    q = torch.cat(q)
    lens = _i32(own)
    out, lse = fm.paged_gqa_decode_shared(q, *caches, _i32(ptable), _i32([prompt]), _i32([0, 4]), _i32(otable), lens, scale,
                                          scale)
    front = fm.paged_cross_attention(q, *caches, _i32(ptable), _i32([prompt]), scale, scale, q_starts=_i32([0, 4]))
    back = fm.paged_cross_attention(q, *caches, _i32(otable), lens, scale, scale)
    joined = fm.attention_merge([front[0], back[0]], [front[1], back[1]])
    want = inputs.ragged.shared(q.cpu().unsqueeze(1), caches[0].cpu(), caches[1].cpu(), ptable, [prompt], [0, 4], otable, own,
                                unit, unit, hd ** -0.5)
    assert fm.last_device_error() == 0
    wrong = inputs.within(out, lse, want, 140)
    assert wrong is None, wrong
    # the merge takes parts that are rounded to bf16 (2^-8 each of sum p |v|) beside what it rounds itself
    assert np.all(np.abs(joined[0].double().cpu().numpy() - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -7 * want[2])
    assert np.all(np.abs(joined[1].double().cpu().numpy() - want[1]) <= inputs.tolerance(want, 140)[1] + 2.0 ** -18)
