"""Append to a paged cache with the rotation on the way, and reading rows back,
on the GPU against the oracle.  Codes and scales are decided in float32 on both
sides (from the same float32 table), so every comparison is bit-exact."""

import numpy as np
import pytest
import torch

import paged_decode_attention_fp8_gb300 as fm
from oracle import fp4
from oracle.attention import e4m3_decode
from oracle.cache_write import quantise_rows, row_inverse, row_scale
from oracle.rotary import rotate_f32

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
SENTINEL = 0x5A


def _rows(seed, shape):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-4, 5, shape[:2] + (1,), generator=g).float())
    return x.to(torch.bfloat16)


def _slots(seed, n, blocks, page, pad=0):
    rng = np.random.default_rng(seed)
    slots = rng.permutation(blocks * page)[:n].astype(np.int32)
    if pad:
        slots[rng.permutation(n)[:pad]] = -1 - rng.integers(0, 5, pad)
    return torch.from_numpy(slots)


def _bf16(x):
    return torch.from_numpy(np.asarray(x)).float().to(torch.bfloat16)


class Caches:
    """K and V caches of one kind with every byte set, on the device, and the oracle's copies."""

    def __init__(self, kind, blocks, h_kv, page, hd, scale=None):
        self.kind, self.hd, self.page = kind, hd, page
        wide = hd // 2 if kind == "fp4" else hd
        self.codes = [np.full((blocks, h_kv, page, wide), SENTINEL, np.uint8) for _ in range(2)]
        self.blocks = [np.full((blocks, h_kv, page, hd // 16), SENTINEL, np.uint8) for _ in range(2)]
        self.rows = [np.full((blocks, h_kv, page), -3.0, np.float32) for _ in range(2)]
        self.scale = scale
        self.dev = [torch.from_numpy(c).to(DEV) for c in self.codes]
        self.dev_blocks = [torch.from_numpy(c).to(DEV) for c in self.blocks]
        self.dev_rows = [torch.from_numpy(c).to(DEV) for c in self.rows]
        self.dev_scale = None if scale is None else [torch.tensor([s], device=DEV) for s in scale]

    def kwargs(self, both=True):
        out = {}
        for i, name in enumerate(("k", "v")[:2 if both else 1]):
            if self.kind == "rows":
                out[name + "_row_scales"] = self.dev_rows[i]
            else:
                out[name + "_scale"] = self.dev_scale[i]
            if self.kind == "fp4":
                out[name + "_block_scales"] = self.dev_blocks[i].view(torch.float8_e4m3fn)
        return out

    def write(self, i, x, slots):
        """The oracle's write of float32 rows x [n, h, hd] into side i."""
        for t, s in enumerate(slots.tolist()):
            if s < 0 or s >= self.codes[i].shape[0] * self.page:
                continue
            at = (s // self.page, slice(None), s % self.page)
            if self.kind == "fp4":
                self.codes[i][at], self.blocks[i][at] = fp4.quantise(x[t], self.scale[i])
            elif self.kind == "rows":
                amax = np.abs(x[t]).max(axis=1).astype(np.float32)
                lift, inv = row_inverse(amax)
                self.rows[i][at] = row_scale(amax)
                self.codes[i][at] = quantise_rows(x[t], inv[:, None], lift[:, None])
            else:
                self.codes[i][at] = quantise_rows(x[t], np.float32(1.0) / np.float32(self.scale[i]))

    def check(self):
        torch.cuda.synchronize()
        for i in range(2):
            assert np.array_equal(self.dev[i].cpu().numpy(), self.codes[i])
            assert np.array_equal(self.dev_blocks[i].cpu().numpy(), self.blocks[i])
            assert np.array_equal(self.dev_rows[i].cpu().numpy(), self.rows[i])


CASES = [  # kind, n, h_q, h_kv, hd, page, rot, offset, interleaved
    ("tensor", 1, 4, 1, 128, 16, 128, 0, False),
    ("rows", 67, 32, 8, 128, 16, 128, 0, False),
    ("fp4", 67, 32, 8, 128, 16, 128, 0, False),
    ("fp4", 33, 0, 3, 64, 32, 64, 0, True),
    ("fp4", 33, 6, 3, 64, 64, 32, 32, False),
    ("fp4", 21, 2, 2, 256, 16, 128, 64, False),
    ("fp4", 21, 2, 2, 96, 16, 48, 16, True),
    ("rows", 40, 5, 5, 80, 48, 80, 0, False),
    ("tensor", 40, 2, 1, 192, 16, 48, 24, False),
    ("rows", 9, 1, 1, 16, 16, 16, 0, False),
    ("tensor", 9, 1, 1, 32, 1, 16, 16, True),
    ("fp4", 30, 1, 1, 1024, 16, 1024, 0, False),
    ("rows", 30, 3, 2, 576, 16, 64, 512, True),
    ("fp4", 30, 3, 2, 576, 64, 64, 512, False),
    ("rows", 5, 1, 1, 512, 16, 512, 0, False),
    ("fp4", 17, 0, 2, 16, 16, 16, 0, True),
]


@pytest.mark.parametrize("kind,n,h_q,h_kv,hd,page,rot,offset,interleaved", CASES)
def test_append_and_read(kind, n, h_q, h_kv, hd, page, rot, offset, interleaved):
    blocks = -(-n // page) + 2
    f, factor = fm.rotary_frequencies(rot, scaling=dict(type="yarn", factor=4, trained=512))
    table = fm.rotary_table(f, 3000, factor=factor)
    k, v = _rows(1, (n, h_kv, hd)), _rows(2, (n, h_kv, hd))
    if n > 8:
        v[3] = 0                      # a zero row
        k[4], v[4] = k[4] * 2.0 ** -80, v[4] * 2.0 ** -80
    slots = _slots(3, n, blocks, page, pad=n // 6)
    pos = torch.randint(0, 3000, (n,), generator=torch.Generator().manual_seed(4))
    if n > 5:
        pos[5] = -1                   # a padded token: nothing of it is written
    q = _rows(5, (n, h_q, hd)) if h_q else None
    c = Caches(kind, blocks, h_kv, page, hd, None if kind == "rows" else (0.0131, 0.0177))
    q_out = torch.full((n, h_q, hd), 9.0, dtype=torch.bfloat16, device=DEV) if h_q else None
    got = fm.paged_kv_append(k.to(DEV), v.to(DEV), slots.to(DEV), c.dev[0], c.dev[1], positions=pos.to(DEV),
                             table=table, interleaved=interleaved, rot_offset=offset,
                             q=None if q is None else q.to(DEV), q_out=q_out, **c.kwargs())
    live = torch.where(pos >= 0, slots, torch.full_like(slots, -1))
    tab = table.cpu().numpy()
    at = pos.clamp(min=0)
    c.write(0, rotate_f32(k, at, tab, interleaved=interleaved, offset=offset), live)
    c.write(1, v.float().numpy(), live)
    c.check()
    if h_q:
        assert got is q_out
        want = _bf16(rotate_f32(q, at, tab, interleaved=interleaved, offset=offset))
        want[pos < 0] = 9.0
        assert torch.equal(q_out.cpu(), want)
    else:
        assert got is None
    # rows read back: the float32 product of value and scale, rounded once
    for i in range(2):
        kw = {n_[2:]: v_ for n_, v_ in c.kwargs().items() if n_.startswith(("k_", "v_")[i])}
        back = fm.paged_cache_read(c.dev[i], live.to(DEV), **kw).cpu()
        for t, s in enumerate(live.tolist()):
            if s < 0:
                assert torch.all(back[t] == 0)
                continue
            row = (s // page, slice(None), s % page)
            if kind == "fp4":
                unit = (e4m3_decode(c.blocks[i][row]).astype(np.float32) * np.float32(c.scale[i])).astype(np.float32)
                val = fp4.dequantise(c.codes[i][row], np.full(c.blocks[i][row].shape, 0x38, np.uint8))
                x = val.astype(np.float32) * np.repeat(unit, 16, axis=-1)
            else:
                unit = c.rows[i][row][:, None] if kind == "rows" else np.float32(c.scale[i])
                x = e4m3_decode(c.codes[i][row]).astype(np.float32) * unit
            assert torch.equal(back[t], _bf16(x.astype(np.float32)))
    assert fm.last_device_error() == 0


def test_without_rotation_equals_the_cache_write():
    """No table: E4M3 rows are the bytes paged_cache_write gives, for K and V in one launch."""
    for kind, scale in (("rows", None), ("tensor", (0.02, 0.03))):
        c, d = (Caches(kind, 7, 4, 16, 128, scale) for _ in range(2))
        k, v = _rows(11, (90, 4, 128)).to(DEV), _rows(12, (90, 4, 128)).to(DEV)
        slots = _slots(13, 90, 7, 16, pad=4).to(DEV)
        assert fm.paged_kv_append(k, v, slots, c.dev[0], c.dev[1], **c.kwargs()) is None
        for i, x in enumerate((k, v)):
            fm.paged_cache_write(x, slots, d.dev[i], tensor_scale=None if kind == "rows" else d.dev_scale[i],
                                 token_scales=d.dev_rows[i] if kind == "rows" else None)
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(c.dev[i], d.dev[i]) and torch.equal(c.dev_rows[i], d.dev_rows[i])


def test_latent_cache_form_and_strides():
    """The dense MLA cache [pages, 64, 576]: k [n, 576], its last 64 dims turned, no V; then rows as
    slices of a projection."""
    f, _ = fm.rotary_frequencies(64)
    table = fm.rotary_table(f, 500)
    n = 150
    wide = _rows(21, (n, 3, 576))
    pos, slots = torch.arange(n, dtype=torch.int32) + 300, _slots(22, n, 4, 64)
    want = Caches("tensor", 4, 1, 64, 576, (0.05, 0.05))
    want.write(0, rotate_f32(wide[:, 1:2], pos, table.cpu().numpy(), interleaved=True, offset=512), slots)
    for x in (wide[:, 1].contiguous().to(DEV), wide.to(DEV)[:, 1], wide.to(DEV)[:, 1:2]):
        cache = torch.full((4, 64, 576), SENTINEL, dtype=torch.uint8, device=DEV)
        fm.paged_kv_append(x, None, slots.to(DEV), cache.view(torch.float8_e4m3fn), positions=pos.to(DEV), table=table,
                           interleaved=True, rot_offset=512, k_scale=torch.tensor([0.05], device=DEV))
        assert np.array_equal(cache.cpu().numpy(), want.codes[0][:, 0])
    back = fm.paged_cache_read(cache, slots.to(DEV), scale=torch.tensor([0.05], device=DEV))
    assert back.shape == (n, 1, 576)
    assert fm.last_device_error() == 0


def test_many_rows_walk_the_grid():
    """More rows than one pass of the grid takes, every token of a batch once."""
    n, h_kv = 6000, 8
    f, _ = fm.rotary_frequencies(128)
    table = fm.rotary_table(f, 8192)
    k, v = _rows(31, (n, h_kv, 128)), _rows(32, (n, h_kv, 128))
    slots = _slots(33, n, 380, 16)
    pos = torch.arange(n, dtype=torch.int32)
    c = Caches("fp4", 380, h_kv, 16, 128, (0.013, 0.011))
    fm.paged_kv_append(k.to(DEV), v.to(DEV), slots.to(DEV), c.dev[0], c.dev[1], positions=pos.to(DEV), table=table,
                       **c.kwargs())
    pick = torch.from_numpy(np.random.default_rng(34).permutation(n)[:300])
    got = [x.cpu().numpy() for x in c.dev + c.dev_blocks]
    x = rotate_f32(k[pick], pos[pick], table.cpu().numpy())
    for side, y in ((0, x), (1, v[pick].float().numpy())):
        codes, s8 = fp4.quantise(y, c.scale[side])
        at = slots[pick].numpy()
        assert np.array_equal(got[side][at // 16, :, at % 16], codes)
        assert np.array_equal(got[2 + side][at // 16, :, at % 16], s8)
    untouched = np.ones(380 * 16, bool)
    untouched[slots.numpy()] = False
    left = got[0].transpose(0, 2, 1, 3).reshape(380 * 16, -1)[untouched]
    assert np.all(left == SENTINEL)


@pytest.mark.parametrize("rot,interleaved", [(0, False), (64, False), (64, True)])
def test_nan_and_infinity_in_four_bits(rot, interleaved):
    """E2M1 has no NaN, so a NaN makes its block's scale NaN (with its partner's block where it is turned) and no other
    block changes; an infinity is stored as the largest value, 448 * 6 scales."""
    n, h_kv, hd, scale = 9, 2, 64, (0.01, 0.02)
    k, v = _rows(51, (n, h_kv, hd)), _rows(52, (n, h_kv, hd))
    bad = [(0, 0, 0), (1, 1, 37), (4, 0, 63), (8, 1, 20)]
    slots = _slots(53, n, 2, 16)
    pos = torch.arange(1, n + 1)
    c = Caches("fp4", 2, h_kv, 16, hd, scale)
    table, kw = None, {}
    if rot:
        table = fm.rotary_table(fm.rotary_frequencies(rot)[0], 100)
        kw = dict(positions=pos.to(DEV), table=table, interleaved=interleaved)
    kn, vn = k.clone(), v.clone()
    for at in bad:
        kn[at] = vn[at] = float("nan")
    vn[5, 1, 18] = -float("inf")
    fm.paged_kv_append(kn.to(DEV), vn.to(DEV), slots.to(DEV), c.dev[0], c.dev[1], **kw, **c.kwargs())
    c.write(0, rotate_f32(k, pos, table.cpu().numpy(), interleaved=interleaved) if rot else k.float().numpy(), slots)
    c.write(1, v.float().numpy(), slots)
    got = [[x.cpu().numpy() for x in y] for y in (c.dev, c.dev_blocks)]
    back = [fm.paged_cache_read(c.dev[i], slots.to(DEV), scale=c.dev_scale[i], block_scales=c.dev_blocks[i]).cpu()
            for i in range(2)]
    for i in range(2):
        touched = {(t, h, d // 16) for t, h, d in bad}
        if rot and i == 0:
            touched |= {(t, h, (d ^ 1 if interleaved else (d + rot // 2) % rot) // 16) for t, h, d in bad}
        for t, h, b in sorted(touched):
            s = int(slots[t])
            at = s // 16, h, s % 16
            assert got[1][i][at + (b,)] & 0x7F == 0x7F
            assert torch.all(torch.isnan(back[i][t, h, 16 * b:16 * b + 16]))
            c.blocks[i][at + (b,)] = got[1][i][at + (b,)]
            c.codes[i][at][8 * b:8 * b + 8] = got[0][i][at][8 * b:8 * b + 8]
        assert int(torch.isnan(back[i]).sum()) == 16 * len(touched)
    s = int(slots[5])
    at = s // 16, 1, s % 16
    assert got[1][1][at + (1,)] == 0x7E and got[0][1][at][9] & 0x0F == 0x0F  # 448, and -6
    assert back[1][5, 1, 18] == _bf16(-np.float32(448 * 6) * np.float32(scale[1]))
    c.blocks[1][at + (1,)], c.codes[1][at][8:16] = 0x7E, got[0][1][at][8:16]
    c.check()


def test_bad_slots_and_positions_are_reported():
    f, _ = fm.rotary_frequencies(64)
    table = fm.rotary_table(f, 100)
    c = Caches("fp4", 2, 2, 16, 64, (0.01, 0.01))
    k = _rows(41, (4, 2, 64))
    slots = torch.tensor([3, 32, -1, 5], dtype=torch.int32)
    pos = torch.tensor([7, 8, 9, 100], dtype=torch.int32)
    q = _rows(42, (4, 1, 64)).to(DEV)
    q_out = torch.full_like(q, 5.0)
    fm.paged_kv_append(k.to(DEV), k.to(DEV), slots.to(DEV), c.dev[0], c.dev[1], positions=pos.to(DEV), table=table,
                       q=q, q_out=q_out, **c.kwargs())
    torch.cuda.synchronize()
    assert fm.last_device_error() == fm.DEV_BAD_SLOT | fm.DEV_BAD_POSITION
    c.write(0, rotate_f32(k[:1], pos[:1], table.cpu().numpy()), slots[:1])
    c.write(1, k[:1].float().numpy(), slots[:1])
    c.check()
    assert torch.all(q_out[3] == 5.0)
    assert torch.equal(q_out[:3].cpu(), _bf16(rotate_f32(q[:3].cpu(), pos[:3], table.cpu().numpy())))
    got = fm.paged_cache_read(c.dev[0], torch.tensor([32, -1, 3], dtype=torch.int32, device=DEV),
                              scale=c.dev_scale[0], block_scales=c.dev_blocks[0])
    torch.cuda.synchronize()
    assert fm.last_device_error() == fm.DEV_BAD_SLOT
    assert torch.all(got[:2] == 0) and torch.any(got[2] != 0)


@pytest.mark.parametrize("kind", ["tensor", "rows"])
@pytest.mark.parametrize("hd", [8, 24, 136, 1024])
def test_read_of_odd_widths(kind, hd):
    """E4M3 rows of any multiple of 8, every code, against the table."""
    rng = np.random.default_rng(51)
    blocks, h_kv, page, n = 5, 3, 16, 70
    codes = rng.integers(0, 256, (blocks, h_kv, page, hd)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x7E
    slots = _slots(52, n, blocks, page, pad=5)
    scales = rng.uniform(0.01, 2.0, (blocks, h_kv, page)).astype(np.float32)
    kw = dict(row_scales=torch.from_numpy(scales).to(DEV)) if kind == "rows" else \
        dict(scale=torch.tensor([0.37], device=DEV))
    got = fm.paged_cache_read(torch.from_numpy(codes).to(DEV), slots.to(DEV), **kw).cpu()
    s = slots.numpy()
    val = e4m3_decode(codes[s // page, :, s % page]).astype(np.float32)
    unit = scales[s // page, :, s % page][..., None] if kind == "rows" else np.float32(0.37)
    want = np.where((s >= 0)[:, None, None], val * unit, 0).astype(np.float32)
    assert torch.equal(got, _bf16(want))
    assert fm.last_device_error() == 0


@pytest.mark.skipif(not hasattr(torch, "float4_e2m1fn_x2"), reason="torch has no packed 4-bit type")
def test_packed_4_bit_type_is_the_same_bytes():
    c, d = (Caches("fp4", 3, 2, 16, 64, (0.01, 0.012)) for _ in range(2))
    k, slots = _rows(71, (20, 2, 64)).to(DEV), _slots(72, 20, 3, 16).to(DEV)
    fm.paged_kv_append(k, k, slots, c.dev[0], c.dev[1], **c.kwargs())
    typed = [x.view(torch.float4_e2m1fn_x2) for x in d.dev]
    fm.paged_kv_append(k, k, slots, typed[0], typed[1], **d.kwargs())
    for i in range(2):
        assert torch.equal(c.dev[i], d.dev[i]) and torch.equal(c.dev_blocks[i], d.dev_blocks[i])
    a = fm.paged_cache_read(c.dev[0], slots, scale=c.dev_scale[0], block_scales=c.dev_blocks[0])
    b = fm.paged_cache_read(typed[0], slots, scale=d.dev_scale[0], block_scales=d.dev_blocks[0])
    assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Slots whose byte offset in the cache passes 2^32 land there, and nowhere else."""
    blocks, h_kv, page, hd = 70000, 8, 64, 128  # 4.6 GB of E4M3 codes
    cache = torch.zeros((blocks, h_kv, page, hd), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((blocks, h_kv, page), device=DEV)
    k = _rows(61, (3, h_kv, hd)).to(DEV)
    slots = torch.tensor([blocks * page - 1, 65536 * page, 5], dtype=torch.int32, device=DEV)
    fm.paged_kv_append(k, None, slots, cache, k_row_scales=scales)
    back = fm.paged_cache_read(cache, slots, row_scales=scales)
    s = slots.long()
    assert int((scales != 0).sum()) == 3 * h_kv
    want = cache.view(torch.float8_e4m3fn)[s // page, :, s % page].float() * scales[s // page, :, s % page][..., None]
    assert torch.equal(back, want.to(torch.bfloat16)) and torch.all(back.abs().amax(-1) > 0)
    # half a step of E4M3 of the row's largest value, 2^-4, and of bf16
    assert torch.all((back.float() - k.float()).abs() <= k.float().abs().amax(-1, keepdim=True) * (2.0 ** -4 + 2.0 ** -8))


def test_wrapper_refusals():
    c = Caches("fp4", 2, 2, 16, 64, (0.01, 0.01))
    e = Caches("tensor", 2, 2, 16, 64, (0.01, 0.01))
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device=DEV)
    slots = torch.arange(4, dtype=torch.int32, device=DEV)
    f, _ = fm.rotary_frequencies(64)
    table = fm.rotary_table(f, 8)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    ok = dict(k=k, v=k, slot_mapping=slots, k_cache=c.dev[0], v_cache=c.dev[1], **c.kwargs())
    fm.paged_kv_append(**ok)
    for bad in [dict(k=k.float()), dict(k=k.cpu()), dict(k=k[..., ::2]), dict(v=k[:3]), dict(v=None),
                dict(slot_mapping=slots.long()), dict(slot_mapping=slots[:2]), dict(k_cache=c.dev[0][:, :1]),
                dict(k_cache=e.dev[0]), dict(v_cache=e.dev[1]), dict(k_scale=None), dict(v_block_scales=None),
                dict(k_scale=torch.zeros(2, device=DEV)), dict(k_row_scales=c.dev_rows[0]),
                dict(k_block_scales=c.dev_blocks[0][..., :2]), dict(q=k), dict(q_out=k), dict(table=table), dict(positions=pos),
                dict(table=table, positions=pos.float()), dict(table=table, positions=pos, q=k, q_out=k[:, :1]),
                dict(table=table.double(), positions=pos)]:
        with pytest.raises(ValueError):
            fm.paged_kv_append(**{**ok, **bad})
    with pytest.raises(fm.FP8MLAError):
        fm.paged_kv_append(**{**ok, "table": table, "positions": pos, "rot_offset": 16})
    with pytest.raises(fm.FP8MLAError) as err:
        fm.paged_kv_append(k, None, slots, e.dev[0].view(torch.float8_e5m2), k_scale=e.dev_scale[0])
    assert err.value.status == 2
    for bad in [dict(cache=c.dev[0].cpu()), dict(slots=slots.long()), dict(scale=None), dict(row_scales=c.dev_rows[0]),
                dict(block_scales=c.dev_blocks[0][:1]), dict(out=k.float())]:
        with pytest.raises(ValueError):
            fm.paged_cache_read(**{**dict(cache=c.dev[0], slots=slots, scale=c.dev_scale[0],
                                          block_scales=c.dev_blocks[0]), **bad})
    # nothing to do is not an error
    assert fm.paged_kv_append(k[:0], k[:0], slots[:0], c.dev[0], c.dev[1], **c.kwargs()) is None
    assert fm.paged_cache_read(e.dev[0], slots[:0], scale=e.dev_scale[0]).shape == (0, 2, 64)
    assert fm.last_device_error() == 0
