"""A prompt appended, then tokens rotated, appended and attended to, against a reference that shares nothing with the
device: the rows turned by the definition, quantised by the oracle and attended to in float64.

Bounds, before any run.  The reference quantises from float32 with the device's own decisions (table entries, the
rotation's two products and sum, the codes), so it holds the cache's values and the rotated query's.  What differs is
the attention: over 4 bits 2^-8 of the output, and of sum p |v| the weights' 2^-11 and 2^-9 for scores, an LSE 2^-12
off; over E4M3 rows this repository's bounds for 16-bit dots (a row's 3e-2, an LSE's 2e-3).  The bounds tell the right
step from a wrong one: the first test puts each mistake into the reference and finds it outside them, on the CPU."""

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from oracle import fp4
from oracle.attention import e4m3_decode, softmax_attention
from oracle.cache_write import quantise_rows, row_inverse, row_scale
from oracle.rotary import rotate_f32
from tests.parity import TOL

H_KV, GROUP, HD, PAGE, BLOCKS = 2, 4, 128, 16, 40
LENS, STEPS, N_POS = [150, 37, 1], 3, 1024
SCALE = {"k": 0.002, "v": 0.0025}
MISTAKES = ["unrotated", "layout", "early", "heads", "missing", "values"]


def _projections():
    """The prompts' and then the steps' rows: lists of bf16 [n, GROUP H_KV + 2 H_KV, HD], one a sequence or a step."""
    rng = np.random.default_rng(5)
    return [torch.from_numpy(rng.standard_normal((n, (GROUP + 2) * H_KV, HD))).to(torch.bfloat16)
            for n in LENS + [len(LENS)] * STEPS]


def _split(x):
    return x[:, :GROUP * H_KV], x[:, GROUP * H_KV:(GROUP + 1) * H_KV], x[:, (GROUP + 1) * H_KV:]


def _host_table():
    f, factor = fm.rotary_frequencies(HD, scaling=dict(type="yarn", factor=4, trained=64))
    angle = np.arange(N_POS)[:, None] * f.numpy()[None, :]
    return np.stack((factor * np.cos(angle), factor * np.sin(angle)), -1).astype(np.float32)


def _quantised(kind, x, side):
    """What the cache stands for after rows x (float32) were written."""
    if kind == "fp4":
        return fp4.dequantise(*fp4.quantise(x, SCALE[side]), float(np.float32(SCALE[side])))
    amax = np.abs(x).max(-1).astype(np.float32)
    lift, inv = row_inverse(amax)
    return e4m3_decode(quantise_rows(x, inv[..., None], lift[..., None])) * row_scale(amax)[..., None].astype(np.float64)


def _reference(kind, interleaved, mistake=None):
    """Per step (out, LSE, sum p |v|, rotated queries) of the step done right, or with a mistake."""
    rows, table = _projections(), _host_table()

    def turn(x, pos):
        if mistake == "unrotated":
            return x.float().numpy()
        return rotate_f32(x, np.maximum(np.asarray(pos) - (mistake == "early"), 0), table,
                          interleaved=interleaved != (mistake == "layout"))

    bs = len(LENS)
    keys, vals = [], []
    for b, n in enumerate(LENS):
        _, k, v = _split(rows[b])
        keys.append(_quantised(kind, turn(k, np.arange(n)), "k"))
        vals.append(_quantised(kind, v.float().numpy(), "v"))
    steps = []
    for step in range(STEPS):
        q, k, v = _split(rows[bs + step])
        now = np.array(LENS) + step
        k, v = _quantised(kind, turn(k, now), "k"), _quantised(kind, v.float().numpy(), "v")
        q = torch.from_numpy(rotate_f32(q, now, table, interleaved=interleaved)).to(torch.bfloat16)
        o, a = (np.zeros((bs, GROUP * H_KV, HD)) for _ in range(2))
        lse = np.zeros((bs, GROUP * H_KV))
        for b in range(bs):
            keys[b], vals[b] = np.concatenate((keys[b], k[b:b + 1])), np.concatenate((vals[b], v[b:b + 1]))
            kk, vv = keys[b], vals[b]
            if mistake == "heads":
                kk = kk[:, ::-1]
            if mistake == "missing":
                kk, vv = kk[:-1], vv[:-1]
            if mistake == "values":
                vv = np.roll(vv, 1, 0)
            for h in range(GROUP * H_KV):
                s = kk[:, h // GROUP] @ q[b, h].double().numpy() * HD ** -0.5
                o[b, h], lse[b, h] = softmax_attention(s, vv[:, h // GROUP])
                a[b, h], _ = softmax_attention(s, np.abs(vv[:, h // GROUP]))
        steps.append((o, lse, a, q))
    return steps


def _off(kind, out, lse, want):
    """How far each row [bs, heads] is off, in units of its bounds."""
    o, l, a, _ = want
    if kind == "fp4":
        tol = 2.0 ** -8 * np.abs(o) + a * (2.0 ** -11 + 2.0 ** -9)  # 0 where every V is
        far = (np.abs(out - o) / np.where(tol > 0, tol, 1e-30)).max(-1)
        return np.maximum(far, np.abs(lse - l) / 2.0 ** -12)
    far = np.linalg.norm(out - o, axis=-1) / np.linalg.norm(o, axis=-1) / TOL["bf16"]["row_rel_l2"]
    return np.maximum(far, np.abs(lse - l) / TOL["bf16"]["lse"])


@pytest.mark.parametrize("kind", ["fp4", "rows"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("mistake", MISTAKES)
def test_the_bounds_exclude_each_mistake(kind, interleaved, mistake):
    for want, wrong in zip(_reference(kind, interleaved), _reference(kind, interleaved, mistake)):
        off = _off(kind, wrong[0], wrong[1], want)
        assert (off > 1).mean() > 0.6 and off.max() > 10
        assert _off(kind, want[0], want[1], want).max() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp4", "rows"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_prompt_then_tokens(kind, interleaved):
    dev, rows, bs = torch.device("cuda"), _projections(), len(LENS)
    bt = np.random.default_rng(6).permutation(BLOCKS)[:bs * 12].reshape(bs, 12).astype(np.int32)
    f, factor = fm.rotary_frequencies(HD, scaling=dict(type="yarn", factor=4, trained=64))
    table = fm.rotary_table(f, N_POS, factor=factor)
    shape = (BLOCKS, H_KV, PAGE)
    kc, vc = (torch.zeros(shape + (HD // 2 if kind == "fp4" else HD,), dtype=torch.uint8, device=dev) for _ in range(2))
    if kind == "fp4":
        kw = dict(k_block_scales=torch.zeros(shape + (HD // 16,), dtype=torch.uint8, device=dev),
                  v_block_scales=torch.zeros(shape + (HD // 16,), dtype=torch.uint8, device=dev),
                  k_scale=torch.tensor([SCALE["k"]], device=dev), v_scale=torch.tensor([SCALE["v"]], device=dev))
    else:
        kw = dict(k_row_scales=torch.ones(shape, device=dev), v_row_scales=torch.ones(shape, device=dev))
    kw.update(table=table, interleaved=interleaved)

    def slots(b, j):
        return (bt[b, j // PAGE] * PAGE + j % PAGE).astype(np.int32)

    for b, n in enumerate(LENS):
        _, k, v = _split(rows[b].to(dev))
        fm.paged_kv_append(k, v, torch.from_numpy(slots(b, np.arange(n))).to(dev), kc, vc,
                           positions=torch.arange(n, device=dev), **kw)
    block_table, seqlens = torch.from_numpy(bt).to(dev), torch.tensor(LENS, dtype=torch.int32, device=dev)
    for step, want in enumerate(_reference(kind, interleaved)):
        q, k, v = _split(rows[bs + step].to(dev))
        now = np.array(LENS) + step
        at = torch.tensor([slots(b, now[b]) for b in range(bs)], dtype=torch.int32, device=dev)
        q = fm.paged_kv_append(k, v, at, kc, vc, positions=torch.from_numpy(now).to(dev), q=q, **kw)
        seqlens += 1
        if kind == "fp4":
            out, lse = fm.paged_gqa_decode_fp4(q, kc, vc, kw["k_block_scales"], kw["v_block_scales"], block_table,
                                               seqlens, kw["k_scale"], kw["v_scale"])
        else:
            out, lse = (t[:, 0] for t in fm.paged_gqa_decode_ext(q.unsqueeze(1), kc, vc, block_table, seqlens,
                                                                 kw["k_row_scales"], kw["v_row_scales"]))
        assert fm.last_device_error() == 0
        assert torch.equal(q.cpu(), want[3])
        assert _off(kind, out.double().cpu().numpy(), lse.double().cpu().numpy(), want).max() <= 1
