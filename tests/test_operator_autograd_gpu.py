"""The rotation inside a torch.autograd.Function, and in-place results seen by autograd."""

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from oracle.rotary import rotate

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


class Rotation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, table):
        ctx.save_for_backward(positions, table)
        return fm.rotary_apply(q, k, positions, table)

    @staticmethod
    def backward(ctx, dq, dk):
        dq, dk = fm.rotary_apply(dq, dk, *ctx.saved_tensors, inverse=True)
        return dq, dk, None, None


def test_gradients_through_a_function():
    """sum(w * rotate(x)^2 / 2): its gradient is the inverse rotation of w * rotate(x), and agrees with differences."""
    rng = np.random.default_rng(1)
    f, factor = fm.rotary_frequencies(32, scaling=dict(type="yarn", factor=4, trained=64))
    table = fm.rotary_table(f, 128, factor=factor)
    pos = np.array([0, 5, 127])
    x = [rng.standard_normal((3, h, 32)).astype(np.float32) for h in (4, 2)]
    w = [rng.standard_normal(v.shape).astype(np.float32) for v in x]
    leaves = [torch.from_numpy(v).to(DEV).requires_grad_() for v in x]
    ys = Rotation.apply(*leaves, torch.from_numpy(pos).to(DEV), table)
    sum((torch.from_numpy(c).to(DEV) * y * y).sum() / 2 for c, y in zip(w, ys)).backward()

    def loss(x):
        return sum(float((c * rotate(v, pos, f, factor=factor) ** 2).sum()) / 2 for c, v in zip(w, x))

    for i in range(2):
        turned = w[i] * rotate(x[i], pos, f, factor=factor)
        want = rotate(turned, pos, f, factor=factor, inverse=True)
        # per direction the table's entries are off by half a step (2^-24), a value by its two products and their sum:
        # 4 half steps of twice the largest; the first direction's error passes w and the second
        tol = factor * (4 * 2.0 ** -24 * 2 * np.abs(turned).max() +
                        2 * np.abs(w[i]).max() * 4 * 2.0 ** -24 * factor * 2 * np.abs(x[i]).max() +
                        2.0 ** -24 * np.abs(turned).max())
        got = leaves[i].grad.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol)
        for _ in range(10):
            at = tuple(rng.integers(s) for s in x[i].shape)
            step = [v.astype(np.float64) for v in x]
            step[i][at] += 1.0  # the loss is quadratic: a central difference of any size is its derivative
            up = loss(step)
            step[i][at] -= 2.0
            assert abs(got[at] - (up - loss(step)) / 2) <= tol + 1e-11


def test_autograd_sees_what_a_call_wrote():
    """A tensor that autograd saved and a call then overwrote is not taken for what it was."""
    f, _ = fm.rotary_frequencies(32)
    table, pos = fm.rotary_table(f, 8), torch.arange(4, device=DEV)
    x = torch.randn((4, 2, 32), device=DEV)
    w = torch.ones((4, 2, 32), device=DEV, requires_grad=True)
    y = (w * x).sum()
    fm.rotary_apply(x, None, pos, table, q_out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    before = x._version
    fm.rotary_apply(w.detach(), None, pos, table, q_out=x)
    assert x._version == before + 1
    cache, out = torch.zeros((1, 2, 16, 32), dtype=torch.uint8, device=DEV), torch.zeros((4, 2, 32), device=DEV)
    out = out.to(torch.bfloat16)
    slots, one = torch.arange(4, dtype=torch.int32, device=DEV), torch.ones(1, device=DEV)
    before = cache._version, out._version
    fm.paged_kv_append(x.to(torch.bfloat16), None, slots, cache, k_scale=one)
    fm.paged_cache_read(cache, slots, scale=one, out=out)
    assert (cache._version, out._version) == (before[0] + 1, before[1] + 1)
    with torch.inference_mode():
        z = torch.zeros((4, 2, 32), device=DEV)
    fm.rotary_apply(x, None, pos, table, q_out=z)  # has no version
    assert torch.equal(z, fm.rotary_apply(x, None, pos, table)[0])
