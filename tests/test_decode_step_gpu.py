"""The operators of a decode step together, as they are used: a prompt appended
(keys rotated) to the caches, then tokens one at a time -- rotate and append,
attend -- against attention in float64 over the keys the caches stand for, and
the same through the E4M3 cache and its decode kernel."""

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from oracle import fp4
from oracle.attention import gqa_decode, spec_visible, softmax_attention  # noqa: F401
from oracle.rotary import rotate

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
H_KV, GROUP, HD, PAGE, BLOCKS = 2, 4, 128, 16, 40


def _slots(bt, b, lo, hi):
    j = np.arange(lo, hi)
    return bt[b, j // PAGE] * PAGE + j % PAGE


@pytest.mark.parametrize("kind", ["fp4", "rows"])
def test_prompt_then_tokens(kind):
    rng = np.random.default_rng(1)
    lens, steps = [150, 37, 1], 3
    bs = len(lens)
    bt = np.zeros((bs, 12), np.int32)
    bt[:] = rng.permutation(BLOCKS)[:bs * 12].reshape(bs, 12)
    f, factor = fm.rotary_frequencies(HD, scaling=dict(type="yarn", factor=4, trained=64))
    table = fm.rotary_table(f, 1024, factor=factor)
    shape = (BLOCKS, H_KV, PAGE)
    wide = HD // 2 if kind == "fp4" else HD
    kc, vc = (torch.zeros(shape + (wide,), dtype=torch.uint8, device=DEV) for _ in range(2))
    if kind == "fp4":
        kw = dict(k_block_scales=torch.zeros(shape + (HD // 16,), dtype=torch.uint8, device=DEV),
                  v_block_scales=torch.zeros(shape + (HD // 16,), dtype=torch.uint8, device=DEV),
                  k_scale=torch.tensor([0.002], device=DEV), v_scale=torch.tensor([0.0025], device=DEV))
    else:
        kw = dict(k_row_scales=torch.ones(shape, device=DEV), v_row_scales=torch.ones(shape, device=DEV))

    def projection(n):
        x = torch.from_numpy(rng.standard_normal((n, GROUP * H_KV + 2 * H_KV, HD))).to(torch.bfloat16)
        return x[:, :GROUP * H_KV], x[:, GROUP * H_KV:GROUP * H_KV + H_KV], x[:, GROUP * H_KV + H_KV:]

    keys, vals = [], []  # unquantised, for the size of the quantisation error
    for b, n in enumerate(lens):
        _, k, v = projection(n)
        slots = torch.from_numpy(_slots(bt, b, 0, n).astype(np.int32)).to(DEV)
        fm.paged_kv_append(k.to(DEV), v.to(DEV), slots, kc, vc, positions=torch.arange(n, device=DEV), table=table, **kw)
        keys.append(rotate(k, np.arange(n), f, factor=factor))
        vals.append(v.double().numpy())
    seqlens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    block_table = torch.from_numpy(bt).to(DEV)
    for step in range(steps):
        now = np.array(lens) + step
        q, k, v = projection(bs)
        slots = np.array([_slots(bt, b, now[b], now[b] + 1)[0] for b in range(bs)], np.int32)
        pos = torch.from_numpy(now.astype(np.int32)).to(DEV)
        q_rot = fm.paged_kv_append(k.to(DEV), v.to(DEV), torch.from_numpy(slots).to(DEV), kc, vc, positions=pos,
                                   table=table, q=q.to(DEV), **kw)
        seqlens += 1
        if kind == "fp4":
            out, lse = fm.paged_gqa_decode_fp4(q_rot, kc, vc, kw["k_block_scales"], kw["v_block_scales"], block_table,
                                               seqlens, kw["k_scale"], kw["v_scale"])
        else:
            out, lse = fm.paged_gqa_decode_ext(q_rot.unsqueeze(1), kc, vc, block_table, seqlens, kw["k_row_scales"],
                                               kw["v_row_scales"])
            out, lse = out[:, 0], lse[:, 0]
        torch.cuda.synchronize()
        assert fm.last_device_error() == 0
        # against the caches' own values: bf16's rounding and the probabilities' (f16, or two E4M3 terms: 2^-8),
        # with 2^-9 of room for the scores' float32 sums
        qn = q_rot.cpu().unsqueeze(1)
        if kind == "fp4":
            o, l, a = fp4.gqa_decode(qn, kc.cpu(), vc.cpu(), kw["k_block_scales"].cpu(), kw["v_block_scales"].cpu(), bt,
                                     now + 1, 0.002, 0.0025, HD ** -0.5)
            o, l, a = o[:, 0], l[:, 0], a[:, 0]
            tol = 2.0 ** -8 * np.abs(o) + a * (2.0 ** -11 + 2.0 ** -9)
            assert np.all(np.abs(out.double().cpu().numpy() - o) <= tol)
            assert np.all(np.abs(lse.double().cpu().numpy() - l) <= 2.0 ** -12)
        else:
            o, l = gqa_decode(qn[:, 0], kc.cpu(), vc.cpu(), bt, now + 1, kw["k_row_scales"].cpu().numpy(),
                              kw["v_row_scales"].cpu().numpy(), HD ** -0.5)
            assert np.linalg.norm(out.double().cpu().numpy() - o) <= 1e-2 * np.linalg.norm(o)
        # against the unquantised step: a rounding of K moves a score by at most scale |q| |dk|
        qr = rotate(q, now, f, factor=factor)
        half = 2.0 ** -2 + 2.0 ** -4 if kind == "fp4" else 2.0 ** -4  # of a value: E2M1 above its smallest, or E4M3
        for b in range(bs):
            keys[b] = np.concatenate((keys[b], rotate(k[b:b + 1], now[b:b + 1], f, factor=factor)))
            vals[b] = np.concatenate((vals[b], v[b:b + 1].double().numpy()))
            for h in range(GROUP * H_KV):
                kk, vv = keys[b][:, h // GROUP], vals[b][:, h // GROUP]
                ref, ref_lse = softmax_attention(kk @ qr[b, h] * HD ** -0.5, vv)
                # E2M1's smallest step is a twelfth of a block's largest value: half of it per value
                dk = half * np.abs(kk) + (np.abs(kk).max() / 12 if kind == "fp4" else 0)
                ds = HD ** -0.5 * (dk @ np.abs(qr[b, h])).max() + 2.0 ** -7 * HD ** -0.5 * \
                    (np.abs(kk) @ np.abs(qr[b, h])).max()
                assert abs(float(lse[b, h]) - ref_lse) <= ds + 1e-3


def test_whole_step_in_one_graph():
    """Append (4-bit) and attend captured once, replayed for new tokens: the same as eager calls."""
    rng = np.random.default_rng(2)
    bs, blocks = 5, 30
    shape = (blocks, H_KV, PAGE)
    f, _ = fm.rotary_frequencies(HD)
    table = fm.rotary_table(f, 256)

    def fresh():
        return [torch.zeros(shape + (w,), dtype=torch.uint8, device=DEV) for w in (HD // 2, HD // 2, HD // 16, HD // 16)]

    scale = torch.tensor([0.002], device=DEV)
    bt = torch.from_numpy(rng.permutation(blocks).reshape(bs, -1).astype(np.int32)).to(DEV)
    rows = [torch.from_numpy(rng.standard_normal((bs, 12, HD))).to(torch.bfloat16).to(DEV) for _ in range(20)]
    x, pos, sl, slots = rows[0].clone(), torch.zeros(bs, dtype=torch.int32, device=DEV), \
        torch.zeros(bs, dtype=torch.int32, device=DEV), torch.zeros(bs, dtype=torch.int32, device=DEV)

    def step(c, out, lse):
        q = fm.paged_kv_append(x[:, 8:10], x[:, 10:], slots, c[0], c[1], positions=pos, table=table, k_scale=scale,
                               v_scale=scale, k_block_scales=c[2], v_block_scales=c[3], q=x[:, :8])
        fm.paged_gqa_decode_fp4(q, c[0], c[1], c[2], c[3], bt, sl, scale, scale, out=out, lse=lse, num_splits=2)

    def at(i):
        x.copy_(rows[i])
        pos.fill_(i)
        sl.fill_(i + 1)
        slots.copy_(bt[:, i // PAGE] * PAGE + i % PAGE)

    c, d = fresh(), fresh()
    out, lse = torch.zeros((bs, 8, HD), dtype=torch.bfloat16, device=DEV), torch.zeros((bs, 8), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        at(0)
        step(c, out, lse)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(c, out, lse)
    want, want_lse = torch.empty_like(out), torch.empty_like(lse)
    for i in range(20):
        at(i)
        g.replay()
        step(d, want, want_lse)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert all(torch.equal(a, b) for a, b in zip(c, d))
    assert fm.last_device_error() == 0
