"""Rotary positions on the GPU against the float64 definition (oracle.rotary).

Tolerance, per value: the table's entries, the two products and the sum are
each rounded to float32 (relative 2^-24 each, so 3 * 2^-24 of |a| + |b| times
the table's factor), then the result to its type: eps / 2 of its size.
"""

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from oracle.rotary import rotate, rotate_f32

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half the spacing of the smallest numbers, where the relative bound ends (bf16 shares float32's exponents)
SMALLEST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def _x(seed, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def _within(y, x, pos, f, factor, interleaved, offset, inverse=False):
    want = rotate(x, pos, f, factor=factor, interleaved=interleaved, offset=offset, inverse=inverse)
    got = y.detach().cpu().double().numpy()
    size = rotate(x.abs(), np.zeros_like(pos), np.zeros(len(f)), factor=1.0)  # |x|
    half = len(f)
    both = np.zeros_like(size)
    d0 = offset + (2 * np.arange(half) if interleaved else np.arange(half))
    d1 = d0 + (1 if interleaved else half)
    both[..., d0] = both[..., d1] = factor * (size[..., d0] + size[..., d1])
    fp32 = 3 * 2.0 ** -24 * both
    tol = fp32 + HALF_STEP[x.dtype] * (np.abs(want) + fp32) + SMALLEST[x.dtype]
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))


CASES = [  # n, h_q, h_k, hd, rot, offset, interleaved, dtype, scaling
    (1, 1, 1, 128, 128, 0, False, torch.bfloat16, None),
    (1, 32, 8, 128, 128, 0, False, torch.bfloat16, None),
    (37, 5, 1, 64, 64, 0, True, torch.bfloat16, dict(type="linear", factor=8)),
    (130, 40, 8, 96, 96, 0, False, torch.float16, dict(type="bands", factor=8, trained=4096)),
    (17, 3, 3, 80, 80, 0, False, torch.float32, dict(type="yarn", factor=8, trained=4096)),
    (65, 16, 1, 576, 64, 512, True, torch.bfloat16, None),      # the latent row: its last 64 dims
    (9, 7, 2, 256, 64, 64, False, torch.float16, None),         # a part in the middle
    (5, 2, 1, 20, 6, 3, False, torch.bfloat16, None),           # nothing a multiple of 8
    (5, 2, 1, 21, 10, 11, True, torch.float32, None),
    (3, 1, 1, 2, 2, 0, False, torch.float16, None),
    (4, 300, 9, 48, 32, 8, True, torch.bfloat16, None),
    (2, 2, 1, 1024, 1000, 8, False, torch.float32, None),       # more pieces than threads, one at a time
    (2, 1, 1, 8192, 8192, 0, False, torch.bfloat16, None),
]


@pytest.mark.parametrize("n,h_q,h_k,hd,rot,offset,interleaved,dtype,scaling", CASES)
def test_rotation(n, h_q, h_k, hd, rot, offset, interleaved, dtype, scaling):
    f, factor = fm.rotary_frequencies(rot, scaling=scaling)
    table = fm.rotary_table(f, 8192, factor=factor)
    q, k = _x(1, (n, h_q, hd), dtype), _x(2, (n, h_k, hd), dtype)
    pos = torch.randint(0, 8192, (n,), generator=torch.Generator().manual_seed(3))
    pos[0] = 8191
    yq, yk = fm.rotary_apply(q.to(DEV), k.to(DEV), pos.to(torch.int32).to(DEV), table, interleaved=interleaved,
                             rot_offset=offset)
    zq, none = fm.rotary_apply(q.to(DEV), None, pos.to(DEV), table, interleaved=interleaved, rot_offset=offset,
                               inverse=True)
    assert none is None
    _within(yq, q, pos.numpy(), f.numpy(), factor, interleaved, offset)
    _within(yk, k, pos.numpy(), f.numpy(), factor, interleaved, offset)
    _within(zq, q, pos.numpy(), f.numpy(), factor, interleaved, offset, inverse=True)
    assert torch.equal(yq.cpu()[..., :offset], q[..., :offset])
    assert torch.equal(yq.cpu()[..., offset + rot:], q[..., offset + rot:])
    if dtype == torch.float32:  # the decisions that the append kernel takes too
        want = rotate_f32(q, pos, table.cpu().numpy(), interleaved=interleaved, offset=offset)
        assert np.array_equal(yq.cpu().numpy(), want)
    assert fm.last_device_error() == 0


def test_table_at_far_positions():
    """A million positions on, angles are still those of 64 bits: within half a float32 step of the
    definition (2^-24 of at most 1) and the 64-bit angle's own rounding (2^20 * 2^-53)."""
    f, _ = fm.rotary_frequencies(64)
    n = 1 << 20
    table = fm.rotary_table(f, n)
    at = torch.tensor([0, 1, 12345, n - 2, n - 1])
    got = table[at.to(DEV)].cpu().double().numpy()
    angle = at.numpy()[:, None] * f.numpy()
    want = np.stack((np.cos(angle), np.sin(angle)), -1)
    assert np.max(np.abs(got - want)) <= 2.0 ** -25 + 2.0 ** -32


def test_in_place_strided_and_unaligned():
    """q and k as slices of one projection, in place; then slices whose addresses allow no wide access."""
    f, _ = fm.rotary_frequencies(64)
    table = fm.rotary_table(f, 512)
    pos = torch.arange(100, 133, dtype=torch.int32)
    rows = _x(5, (33, 12, 64), torch.bfloat16)
    dev = rows.to(DEV)
    want_q, want_k = fm.rotary_apply(rows[:, :8].contiguous().to(DEV), rows[:, 8:10].contiguous().to(DEV),
                                     pos.to(DEV), table)
    q, k = dev[:, :8], dev[:, 8:10]
    a, b = fm.rotary_apply(q, k, pos.to(DEV), table, q_out=q, k_out=k)
    assert a is q and b is k
    assert torch.equal(dev[:, :8], want_q) and torch.equal(dev[:, 8:10], want_k)
    assert torch.equal(dev[:, 10:].cpu(), rows[:, 10:])  # the values beside them are left alone
    odd = torch.zeros((33, 8, 67), dtype=torch.bfloat16, device=DEV)[..., 3:]
    odd.copy_(rows[:, :8])
    heads_last = torch.empty((8, 33, 64), dtype=torch.bfloat16, device=DEV).transpose(0, 1)  # token stride < head stride
    c, _ = fm.rotary_apply(odd, None, pos.to(DEV), table, q_out=heads_last)
    assert torch.equal(c, want_q)
    assert fm.last_device_error() == 0


def test_padding_and_positions_past_the_table():
    f, _ = fm.rotary_frequencies(32)
    table = fm.rotary_table(f, 64)
    q = _x(6, (6, 2, 32), torch.float32).to(DEV)
    out = torch.full_like(q, -7.0)
    pos = torch.tensor([5, -1, 63, 64, 1 << 40, -(1 << 40)], device=DEV)
    fm.rotary_apply(q, None, pos, table, q_out=out)
    torch.cuda.synchronize()
    assert fm.last_device_error() == fm.DEV_BAD_POSITION
    assert fm.last_device_error() == 0
    for i in (1, 3, 4, 5):
        assert torch.all(out[i] == -7.0)
    _within(out[[0, 2]], q[[0, 2]].cpu(), np.array([5, 63]), f.numpy(), 1.0, False, 0)


def test_inverse_is_the_gradient():
    """d/dx of sum(w * rotate(x)) is the inverse rotation of w: against differences in float64."""
    f, factor = fm.rotary_frequencies(16, scaling=dict(type="yarn", factor=4, trained=64))
    table = fm.rotary_table(f, 128, factor=factor)
    x, w = _x(7, (3, 2, 24), torch.float32), _x(8, (3, 2, 24), torch.float32)
    pos = torch.tensor([1, 77, 127])
    grad, _ = fm.rotary_apply(w.to(DEV), None, pos.to(DEV), table, rot_offset=8, inverse=True)
    rng = np.random.default_rng(9)
    for _ in range(20):
        i, h, d = rng.integers(3), rng.integers(2), rng.integers(24)
        step = np.zeros(x.shape)
        step[i, h, d] = 1.0  # the map is linear: a difference of any size is its derivative
        up = rotate(x.double().numpy() + step, pos, f, factor=factor, offset=8)
        down = rotate(x.double().numpy() - step, pos, f, factor=factor, offset=8)
        want = np.sum(w.double().numpy() * (up - down)) / 2
        # float32 rotation of w (as above), and sums of 144 terms in 64 bits
        tol = 4 * 2.0 ** -24 * factor * 2 * float(w.abs().max()) + 1e-13
        assert abs(float(grad[i, h, d]) - want) <= tol


def test_graph_capture_other_stream_and_empty():
    f, _ = fm.rotary_frequencies(128)
    table = fm.rotary_table(f, 4096)
    q, k = _x(10, (64, 32, 128), torch.bfloat16).to(DEV), _x(11, (64, 8, 128), torch.bfloat16).to(DEV)
    pos = torch.arange(64, dtype=torch.int32, device=DEV)
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    want = fm.rotary_apply(q, k, pos, table)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        fm.rotary_apply(q, k, pos, table, q_out=yq, k_out=yk)
    side.synchronize()
    assert torch.equal(yq, want[0]) and torch.equal(yk, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fm.rotary_apply(q, k, pos, table, q_out=yq, k_out=yk)
    pos += 1000
    g.replay()
    want = fm.rotary_apply(q, k, pos, table)
    assert torch.equal(yq, want[0]) and torch.equal(yk, want[1])
    empty, _ = fm.rotary_apply(q[:0], None, pos[:0], table)
    assert empty.shape == (0, 32, 128)
    assert fm.rotary_table(f, 0).shape == (0, 64, 2)
    assert fm.last_device_error() == 0


def test_wrapper_refusals():
    f, _ = fm.rotary_frequencies(32)
    table = fm.rotary_table(f, 16)
    q = torch.zeros((4, 2, 32), dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    for bad in [dict(q=q.cpu()), dict(q=q.double()), dict(q=q[..., ::2]), dict(k=q[:3]), dict(k=q.float()),
                dict(k=q[..., :16]), dict(positions=pos[:3]), dict(positions=pos.float()), dict(positions=pos.cpu()),
                dict(table=table.double()), dict(table=table[..., 0]), dict(table=table.cpu()),
                dict(q_out=q[:, :1]), dict(q_out=q.float()), dict(k_out=q),
                dict(q_out=q[:1].expand(4, 2, 32)), dict(q_out=q[:, :1].expand(4, 2, 32))]:
        a = dict(q=q, k=None, positions=pos, table=table)
        kw = {n: v for n, v in bad.items() if n.endswith("_out")}
        a.update({n: v for n, v in bad.items() if n not in kw})
        with pytest.raises(ValueError):
            fm.rotary_apply(a["q"], a["k"], a["positions"], a["table"], **kw)
    for kw in (dict(rot_offset=1), dict(rot_offset=-1)):
        with pytest.raises(fm.FP8MLAError):
            fm.rotary_apply(q, None, pos, table, **kw)
    with pytest.raises(ValueError):
        fm.rotary_table(f.float(), 16)
    with pytest.raises(fm.FP8MLAError):
        fm.rotary_table(f, 16, factor=0.0)
