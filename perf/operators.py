"""Cases of the rotary, cache-append, cache-read and 4-bit-cache attention operators.

Each case is one pass through one operator.  ``run`` computes it either in
elementary torch operations (``own`` false) or through the library's public
entry points (``own`` true); both take what ``prepare`` makes.  ``exact``
gives the same outputs from the definitions in 64 bits, written apart from
the plain form.

The 4-bit cache holds E2M1 values (two to a byte, the even dimension in the
low half), one E4M3 scale per 16 values of a row and one float32 scale for
the whole cache: value = E2M1 * block scale * cache scale.
"""

import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# ------------------------------------------------------------------ cases --


def listed():
    rotary = dict(op="rotary", hd=128, rot=128, offset=0, interleaved=False, scaling="none", dtype="bf16")
    append = dict(op="append", h_q=32, h_kv=8, hd=128, page=16, rot=128, offset=0, interleaved=False,
                  scaling="none", kind="rows", values=True, pad=0)
    read = dict(op="read", h_kv=8, hd=128, page=16)
    attend = dict(op="attend", h_kv=8, group=4, hd=128, page=16, q_len=1, window=0, sinks=False, mask=False)
    return [
        # one new token of one sequence: the smallest call, host and launch latency
        dict(rotary, name="rotary one token", n=1, h_q=32, h_k=8, n_pos=16384),
        # a prompt chunk of odd length at far positions of a stretched context
        dict(rotary, name="rotary prompt chunk", n=8191, h_q=32, h_k=8, n_pos=131072, scaling="yarn"),
        # the new token of each of 64 sequences, some slots of the batch empty: a decode step's append
        dict(append, name="append decode step", n=64, pad=5, n_pos=16384),
        # a prompt's K and V into caches with one scale each
        dict(append, name="append prompt", n=16384, h_q=0, kind="tensor", n_pos=131072, scaling="bands"),
        # the latent cache: one 576-wide row a token whose last 64 values are rotated pairwise, with the queries
        dict(append, name="append latent rows", n=2049, h_q=16, h_kv=1, hd=576, page=64, rot=64, offset=512,
             interleaved=True, kind="tensor", values=False, n_pos=65536),
        # a prompt chunk into the 4-bit cache, read back as its prefill attention takes it
        dict(append, name="append 4-bit and read", n=8193, h_q=0, kind="fp4", n_pos=65536),
        # rows of a few shared pages, as a short prefix is reused
        dict(read, name="read short prefix", n=48, kind="fp4"),
        # a long shared prefix out of the cache with a scale per row
        dict(read, name="read long prefix", n=65537, kind="rows"),
        # one sequence with a short context: latency
        dict(attend, name="attend one short", bs=1, lo=777, hi=777),
        # a served batch of unequal contexts
        dict(attend, name="attend batch", bs=32, lo=1024, hi=16384),
        # speculative block of four tokens, sliding window and sinks
        dict(attend, name="attend block window", bs=32, lo=1024, hi=16384, q_len=4, window=4096, sinks=True,
             mask=True),
        # few KV heads, long contexts, narrow heads, larger pages: the split over the keys carries it
        dict(attend, name="attend long narrow", bs=3, lo=50001, hi=131071, h_kv=2, group=8, hd=64, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def _draw_rotary_shape(rng, hd):
    interleaved = rng.random() < 0.4
    rot = hd if rng.random() < 0.6 else (hd // 2 if hd % 64 == 0 else hd)
    offset = 0 if rot == hd or rng.random() < 0.5 else hd - rot
    return dict(rot=rot, offset=offset, interleaved=interleaved,
                scaling=rng.choice(["none", "linear", "bands", "yarn"]), n_pos=_log(rng, 2048, 131072))


def draw(rng):
    op = rng.choice(["rotary", "append", "read", "attend", "attend"])
    if op == "rotary":
        hd = rng.choice([64, 80, 96, 128, 128, 192, 256])
        h_k = rng.choice([1, 2, 4, 8])
        return dict(op=op, n=_log(rng, 1, 8191), h_q=h_k * rng.choice([1, 3, 4]), h_k=h_k, hd=hd,
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), **_draw_rotary_shape(rng, hd))
    if op == "append":
        kind = rng.choice(["tensor", "rows", "fp4", "fp4"])
        hd = rng.choice([64, 128, 128, 256])
        h_kv = rng.choice([1, 2, 4, 8])
        n = _log(rng, 1, 8192)
        return dict(op=op, n=n, h_q=rng.choice([0, h_kv, 4 * h_kv]), h_kv=h_kv, hd=hd, page=rng.choice([16, 32, 64]),
                    kind=kind, values=True, pad=rng.randint(0, n // 4), **_draw_rotary_shape(rng, hd))
    if op == "read":
        return dict(op=op, n=_log(rng, 1, 65536), h_kv=rng.choice([1, 2, 4, 8]), hd=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64]), kind=rng.choice(["tensor", "rows", "fp4", "fp4"]))
    q_len = rng.choice([1, 1, 1, 2, 3, 4])
    group = rng.choice([1, 2, 3, 4, 4, 7, 8, 16])
    while q_len * group > 16:
        q_len -= 1
    bs = _log(rng, 1, 64)
    hi = _log(rng, 1, min(131072, 500000 // bs))
    return dict(op=op, bs=bs, lo=rng.randint(0, hi) if rng.random() < 0.5 else hi, hi=hi,
                h_kv=rng.choice([1, 2, 4, 8]) if hi * bs < 250000 else rng.choice([1, 2, 4]), group=group,
                hd=rng.choice([64, 128, 128, 128]), page=rng.choice([16, 16, 32, 64]), q_len=q_len,
                window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]), sinks=rng.random() < 0.3,
                mask=q_len > 1 and rng.random() < 0.5)


# ----------------------------------------------------------------- inputs --


def _inv_freq(c):
    """Angular frequencies of the rotated pairs (64 bits) and the factor on cos and sin."""
    rot, theta, factor, trained = c["rot"], 10000.0, 8.0, 4096
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if c["scaling"] == "linear":
        return f / factor, 1.0
    if c["scaling"] == "bands":  # long waves are stretched, short ones kept, those between blended
        turns = trained * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 1.0
    if c["scaling"] == "yarn":
        at = [rot * math.log(trained / (b * 2 * math.pi)) / (2 * math.log(theta)) for b in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        keep = 1 - ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _rotary_state(c, g):
    f, factor = _inv_freq(c)
    f = f.cuda()
    angle = torch.arange(c["n_pos"], device="cuda", dtype=torch.float64)[:, None] * f
    table = torch.stack((angle.cos(), angle.sin()), -1).mul_(factor).float()
    first = torch.randint(0, max(1, c["n_pos"] - c["n"]), (1,), device="cuda", generator=g)
    if c["n"] <= 512:  # the new tokens of as many sequences
        positions = torch.randint(0, c["n_pos"], (c["n"],), device="cuda", generator=g)
    else:              # a run of one sequence
        positions = (first + torch.arange(c["n"], device="cuda")) % c["n_pos"]
    return dict(table=table, positions=positions.to(torch.int32), inv_freq=f, factor=factor)


def _rows(g, shape, dtype=torch.bfloat16):
    """Activations of a projection: normal values, some dimensions several times the others."""
    x = torch.randn(shape, device="cuda", generator=g)
    gain = torch.randn(shape[-1], device="cuda", generator=g).mul_(0.5).exp_()
    return (x * gain).to(dtype)


def _pages(g, used, spare):
    return torch.randperm(used + spare, device="cuda", generator=g)[:used]


def _cache_shapes(c, blocks):
    wide = c["hd"] // 2 if c["kind"] == "fp4" else c["hd"]
    return (blocks, c["h_kv"], c["page"], wide), (blocks, c["h_kv"], c["page"], c["hd"] // 16)


def _quantise_fp4(x, scale):
    """E2M1 codes and E4M3 block scales of x [..., hd], in 32 bits throughout."""
    blocks = x.float().unflatten(-1, (-1, 16))
    amax = blocks.abs().amax(-1)
    s8 = (amax * (1.0 / (scale * 6.0))).clamp(max=448.0).to(E4M3)
    s = s8.float()
    inv = torch.where(s > 0, 1.0 / (s * scale), torch.zeros_like(s))
    y = blocks * inv[..., None]
    a = y.abs().clamp(max=6.0)
    near = torch.where(a < 2, (a * 2).round() * 0.5, torch.where(a < 4, a.round(), (a * 0.5).round() * 2))
    mag = torch.where(near < 2, near * 2, torch.where(near < 4, near + 2, near * 0.5 + 4)).to(torch.uint8)
    code = mag | torch.where(torch.signbit(y) & (s > 0)[..., None], 8, 0).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s8


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "rotary":
        s = _rotary_state(c, g)
        rows = _rows(g, (c["n"], c["h_q"] + 2 * c["h_k"], c["hd"]), DTYPES[c["dtype"]])  # one projection's output
        return dict(s, c=c, q=rows[:, :c["h_q"]], k=rows[:, c["h_q"]:c["h_q"] + c["h_k"]])
    if c["op"] == "append":
        s = _rotary_state(c, g)
        n, page = c["n"], c["page"]
        copies = 2 if c["values"] else 1
        rows = _rows(g, (n, c["h_q"] + copies * c["h_kv"], c["hd"]))
        s.update(c=c, q=rows[:, :c["h_q"]] if c["h_q"] else None, k=rows[:, c["h_q"]:c["h_q"] + c["h_kv"]],
                 v=rows[:, c["h_q"] + c["h_kv"]:] if c["values"] else None)
        blocks = -(-n // page) + 3
        perm = torch.randperm(blocks, device="cuda", generator=g)
        t = torch.arange(n, device="cuda")
        slots = perm[t // page] * page + t % page
        if c["pad"]:
            slots[torch.randperm(n, device="cuda", generator=g)[:c["pad"]]] = -1
        s["slots"] = slots.to(torch.int32)
        shape, blocked = _cache_shapes(c, blocks)
        for name in ("k", "v")[:copies]:
            amax = s[name].float().abs().amax() * (1.0 + torch.rand((), device="cuda", generator=g))  # calibrated before
            s[name + "_cache"] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
            if c["kind"] == "rows":
                s[name + "_row_scales"] = torch.ones(shape[:3], device="cuda")
            else:
                s[name + "_scale"] = (amax / (448.0 * 6.0 if c["kind"] == "fp4" else 448.0)).reshape(1)
            if c["kind"] == "fp4":
                s[name + "_blocks"] = torch.zeros(blocked, dtype=torch.uint8, device="cuda").view(E4M3)
        return s
    if c["op"] == "read":
        n, page = c["n"], c["page"]
        blocks = -(-n // page) + 2
        x = _rows(g, (blocks, c["h_kv"], page, c["hd"]))
        s = dict(c=c)
        amax = x.float().abs().amax(-1)
        if c["kind"] == "rows":
            s["row_scales"] = amax / 448.0
            s["cache"] = (x.float() / s["row_scales"][..., None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        elif c["kind"] == "tensor":
            s["scale"] = (amax.amax() / 448.0).reshape(1)
            s["cache"] = (x.float() / s["scale"]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        else:
            s["scale"] = (amax.amax() / (448.0 * 6.0)).reshape(1)
            s["cache"], s["blocks"] = _quantise_fp4(x, s["scale"])
        perm = torch.randperm(blocks, device="cuda", generator=g)
        t = torch.arange(n, device="cuda")
        s["slots"] = (perm[t // page] * page + t % page).to(torch.int32)
        return s
    # attend
    bs, page, h_kv, hd = c["bs"], c["page"], c["h_kv"], c["hd"]
    lens = torch.randint(c["lo"], c["hi"] + 1, (bs,), device="cuda", generator=g)
    lens[0] = c["hi"]
    blocks_of = (lens + page - 1) // page
    most = max(1, -(-c["hi"] // page))
    used = max(1, int(blocks_of.sum()))
    perm = _pages(g, used, 2)
    first = blocks_of.cumsum(0) - blocks_of
    at = torch.arange(most, device="cuda")
    table = perm[(first[:, None] + at).clamp(max=used - 1)]
    table = torch.where(at < blocks_of[:, None], table, torch.zeros_like(table)).to(torch.int32)
    s = dict(c=c, table=table, lens=lens.to(torch.int32), softmax_scale=hd ** -0.5)
    for name in ("k", "v"):
        x = _rows(g, (used + 2, h_kv, page, hd))
        s[name + "_scale"] = (x.abs().amax().float() / (448.0 * 6.0)).reshape(1)
        s[name + "_cache"], s[name + "_blocks"] = _quantise_fp4(x, s[name + "_scale"])
        del x
    q_shape = (bs, c["q_len"], h_kv * c["group"], hd)
    s["q"] = torch.randn(q_shape, device="cuda", generator=g).to(torch.bfloat16)
    s["mask"] = None
    if c["mask"]:  # a tree of drafted tokens: each sees itself and some before it
        m = torch.rand((bs, c["q_len"], c["q_len"]), device="cuda", generator=g) < 0.6
        s["mask"] = (m.tril() | torch.eye(c["q_len"], dtype=torch.bool, device="cuda")).to(torch.uint8)
    s["sinks"] = torch.randn(q_shape[2], device="cuda", generator=g) if c["sinks"] else None
    return s


# ------------------------------------------------------------- plain form --


def _rotate(x, s):
    """x [n, h, hd] in 32 bits with its rotated part turned by the table's angles."""
    c = s["c"]
    cs = s["table"][s["positions"].long()][:, None]
    co, si = cs[..., 0], cs[..., 1]
    x = x.float()
    part = x[..., c["offset"]:c["offset"] + c["rot"]]
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * co - b * si, b * co + a * si), -1).flatten(-2)
    else:
        a, b = part.chunk(2, -1)
        part = torch.cat((a * co - b * si, b * co + a * si), -1)
    return torch.cat((x[..., :c["offset"]], part, x[..., c["offset"] + c["rot"]:]), -1)


def _put(cache, slots, rows):
    """The cache [blocks, h, page, w] with rows [n, h, w] in their slots; a negative slot is left out."""
    blocks, h, page, w = cache.shape
    token = torch.full((blocks * page + 1,), -1, dtype=torch.int64, device=cache.device)
    token[torch.where(slots < 0, blocks * page, slots).long()] = torch.arange(len(slots), device=cache.device)
    token = token[:-1]
    new = rows[token.clamp(min=0)].reshape(blocks, page, h, w).transpose(1, 2)
    cache.copy_(torch.where((token >= 0).reshape(blocks, 1, page, 1), new, cache))


def _plain_append(s):
    c = s["c"]
    for name in ("k", "v") if c["values"] else ("k",):
        x = _rotate(s[name], s) if name == "k" else s[name].float()
        cache = s[name + "_cache"]
        if c["kind"] == "fp4":
            codes, blocks = _quantise_fp4(x, s[name + "_scale"])
            _put(cache, s["slots"], codes)
            _put(s[name + "_blocks"].view(torch.uint8), s["slots"], blocks.view(torch.uint8))
            continue
        if c["kind"] == "rows":
            amax = x.abs().amax(-1)
            one = torch.ones_like(amax)
            inv = torch.where(amax > 0, 448.0 / amax, one)[..., None]
            _put(s[name + "_row_scales"][..., None], s["slots"], torch.where(amax > 0, amax / 448.0, one)[..., None])
        else:
            inv = 1.0 / s[name + "_scale"]
        _put(cache, s["slots"], (x * inv).clamp(-448, 448).to(E4M3).view(torch.uint8))
    return _rotate(s["q"], s).to(torch.bfloat16) if c["h_q"] else None


def _values_fp4(codes, blocks):
    """E2M1 value times block scale of packed codes [..., hd / 2], in 32 bits."""
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return lut[both.int()].unflatten(-1, (-1, 16)), blocks.float()[..., None]


def _plain_read(kind, cache, slots, scale, row_scales, blocks):
    page = cache.shape[2]
    at = slots.clamp(min=0).long()
    block, off = at // page, at % page
    if kind == "fp4":
        e, b = _values_fp4(cache[block, :, off], blocks.view(torch.uint8)[block, :, off].view(E4M3))
        x = (e * (b * scale)).flatten(-2)
    elif kind == "rows":
        x = cache[block, :, off].view(E4M3).float() * row_scales[block, :, off][..., None]
    else:
        x = cache[block, :, off].view(E4M3).float() * scale
    return torch.where((slots >= 0)[:, None, None], x, torch.zeros_like(x)).to(torch.bfloat16)


def _visible(c, lens, mask, keys):
    """[bs, q_len, keys] truth values: which keys each query token sees."""
    j = torch.arange(keys, device=lens.device)[None, None, :]
    start = (lens.long() - c["q_len"])[:, None, None]
    i = torch.arange(c["q_len"], device=lens.device)[None, :, None]
    at = (j - start).expand(len(lens), c["q_len"], keys)
    if mask is None:
        inside = at <= i
    else:
        inside = torch.gather(mask.bool(), 2, at.clamp(0, c["q_len"] - 1))
    see = (j < lens[:, None, None]) & ((at < 0) | inside)
    return see & (i - at < c["window"]) if c["window"] else see


def _plain_attend(s):
    c = s["c"]
    bs, h_kv, group, hd, q_len = c["bs"], c["h_kv"], c["group"], c["hd"], c["q_len"]
    at = s["table"].long()

    def gathered(name):
        e, b = _values_fp4(s[name + "_cache"][at], s[name + "_blocks"].view(torch.uint8)[at].view(E4M3))
        return (e * b).flatten(-2).transpose(1, 2).reshape(bs, h_kv, -1, hd)  # [bs, h_kv, keys, hd]

    k = gathered("k")
    q = s["q"].float().reshape(bs, q_len, h_kv, group, hd).permute(0, 2, 1, 3, 4).reshape(bs, h_kv, -1, hd)
    score = (q @ k.transpose(-1, -2)) * (s["softmax_scale"] * s["k_scale"])
    del k
    see = _visible(c, s["lens"], s["mask"], score.shape[-1])[:, None, :, None]
    score = score.reshape(bs, h_kv, q_len, group, -1)
    score = torch.where(see, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    if c["sinks"]:
        sink = s["sinks"].reshape(1, h_kv, 1, group, 1)
        top = torch.maximum(top, sink)
    top0 = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (score - top0).exp()
    total = p.sum(-1, keepdim=True)
    if c["sinks"]:
        total = total + (sink - top0).exp()
    v = gathered("v")
    o = (p.reshape(bs, h_kv, q_len * group, -1) @ v).reshape(bs, h_kv, q_len, group, hd) * s["v_scale"]
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top0 + total.log())[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(bs, q_len, h_kv * group, hd)
    return o.to(torch.bfloat16), lse.permute(0, 2, 1, 3).reshape(bs, q_len, h_kv * group)


# -------------------------------------------------------------------- run --


def run(state):
    s = state
    c = s["c"]
    if own:
        import paged_decode_attention_fp8_gb300 as fm
    if c["op"] == "rotary":
        if own:
            q, k = fm.rotary_apply(s["q"], s["k"], s["positions"], s["table"], interleaved=c["interleaved"],
                                   rot_offset=c["offset"])
        else:
            q, k = (_rotate(x, s).to(x.dtype) for x in (s["q"], s["k"]))
        return {"q": q, "k": k}
    if c["op"] == "append":
        names = ("k", "v") if c["values"] else ("k",)
        if own:
            q = fm.paged_kv_append(s["k"], s["v"], s["slots"], s["k_cache"], s.get("v_cache"),
                                   positions=s["positions"], table=s["table"], interleaved=c["interleaved"],
                                   rot_offset=c["offset"], k_scale=s.get("k_scale"), v_scale=s.get("v_scale"),
                                   k_row_scales=s.get("k_row_scales"), v_row_scales=s.get("v_row_scales"),
                                   k_block_scales=s.get("k_blocks"), v_block_scales=s.get("v_blocks"), q=s["q"])
        else:
            q = _plain_append(s)
        out = {"q": q} if c["h_q"] else {}
        for name in names:
            if c["kind"] == "fp4":  # what the 4 bits stand for is read back from the cache
                if own:
                    out[name] = fm.paged_cache_read(s[name + "_cache"], s["slots"], scale=s[name + "_scale"],
                                                    block_scales=s[name + "_blocks"])
                else:
                    out[name] = _plain_read("fp4", s[name + "_cache"], s["slots"], s[name + "_scale"], None,
                                            s[name + "_blocks"])
            else:
                out[name] = s[name + "_cache"].view(E4M3)
                if c["kind"] == "rows":
                    out[name + "_row_scales"] = s[name + "_row_scales"]
        return out
    if c["op"] == "read":
        if own:
            return fm.paged_cache_read(s["cache"], s["slots"], scale=s.get("scale"), row_scales=s.get("row_scales"),
                                       block_scales=s.get("blocks"))
        return _plain_read(c["kind"], s["cache"], s["slots"], s.get("scale"), s.get("row_scales"), s.get("blocks"))
    if own:
        out, lse = fm.paged_gqa_decode_fp4(s["q"], s["k_cache"], s["v_cache"], s["k_blocks"], s["v_blocks"],
                                           s["table"], s["lens"], s["k_scale"], s["v_scale"],
                                           softmax_scale=s["softmax_scale"], spec_mask=s["mask"],
                                           window=c["window"], sinks=s["sinks"])
    else:
        out, lse = _plain_attend(s)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------- work --


def _row_bytes(c):
    """Bytes a cached row takes: codes and scales."""
    return {"fp4": c["hd"] / 2 + c["hd"] / 16, "rows": c["hd"] + 4, "tensor": c["hd"]}[c["kind"]]


def work(case):
    c = case
    if c["op"] == "rotary":
        size = 4 if c["dtype"] == "f32" else 2
        heads = c["h_q"] + c["h_k"]
        return {"bytes": c["n"] * (heads * c["hd"] * 2 * size + c["rot"] * 4 + 4),
                "flops": c["n"] * heads * c["rot"] * 3}
    if c["op"] == "append":
        copies = 2 if c["values"] else 1
        written = c["n"] - c["pad"]
        data = written * copies * c["h_kv"] * (c["hd"] * 2 + _row_bytes(c)) + c["n"] * (c["h_q"] * c["hd"] * 4 + 8)
        if c["kind"] == "fp4":  # the read back: codes and scales in, 16-bit values out
            data += written * copies * c["h_kv"] * _row_bytes(c) + c["n"] * copies * c["h_kv"] * c["hd"] * 2
        return {"bytes": data + c["n"] * c["rot"] * 4,
                "flops": c["n"] * (c["h_q"] + c["h_kv"]) * c["rot"] * 3 + written * copies * c["h_kv"] * c["hd"] * 3}
    if c["op"] == "read":
        return {"bytes": c["n"] * (c["h_kv"] * (_row_bytes(c) + c["hd"] * 2) + 4), "flops": c["n"] * c["h_kv"] * c["hd"]}
    # attend: the first sequence has hi keys, the others lie evenly between lo and hi; a window leaves the last ones
    span = c["window"] + c["q_len"] - 1 if c["window"] else c["hi"]
    if c["bs"] == 1 or c["lo"] == c["hi"]:
        keys = c["bs"] * min(c["hi"], span)
    elif span <= c["lo"]:
        keys = c["bs"] * span
    else:
        top = min(span, c["hi"])
        mean = ((top * (top + 1) - c["lo"] * (c["lo"] - 1)) / 2 + (c["hi"] - top) * span) / (c["hi"] - c["lo"] + 1)
        keys = (c["bs"] - 1) * mean + min(c["hi"], span)
    cols = c["q_len"] * c["group"]
    return {"bytes": keys * c["h_kv"] * 2 * (c["hd"] / 2 + c["hd"] / 16) + c["bs"] * c["h_kv"] * cols * (c["hd"] * 4 + 4)
            + c["bs"] * 4 * -(-c["hi"] // c["page"]),
            "flops": keys * c["h_kv"] * cols * c["hd"] * 4}


# ---------------------------------------------------- definition, 64 bits --


def _exact_turn(x, s):
    """Rotation of pairs as multiplication by e^(i angle), angles from the frequencies themselves."""
    c = s["c"]
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]
    turn = torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None, :]
    y = x.double().clone()
    lo, half = c["offset"], c["rot"] // 2
    first = torch.arange(half, device=x.device) * 2 + lo if c["interleaved"] else torch.arange(half, device=x.device) + lo
    second = first + (1 if c["interleaved"] else half)
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real.contiguous(), z.imag.contiguous()
    return y


def _exact_e4m3(x):
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def _exact_e2m1(x):
    a = x.abs()
    grid = [0.5, 0.5, 0.5, 0.5, 1.0, 1.0, 2.0]
    edge = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    y = torch.zeros_like(a)
    for n, (e, w) in enumerate(zip(edge, grid)):  # a tie goes to the even code
        y += w * ((a >= e) if n % 2 else (a > e)).double()
    return torch.sign(x) * y


def _exact_blocks(x, scale):
    b = x.unflatten(-1, (-1, 16))
    s8 = _exact_e4m3(b.abs().amax(-1) / (6.0 * scale))
    d = (s8 * scale)[..., None]
    return (torch.where(d > 0, _exact_e2m1(torch.where(d > 0, b / d, b)), torch.zeros_like(b)) * d).flatten(-2)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rotary":
        return {"q": _exact_turn(s["q"], s), "k": _exact_turn(s["k"], s)}
    if c["op"] == "append":
        out = {"q": _exact_turn(s["q"], s)} if c["h_q"] else {}
        live = (s["slots"] >= 0).nonzero()[:, 0]
        at = s["slots"][live].long()
        block, off = at // c["page"], at % c["page"]
        for name in ("k", "v") if c["values"] else ("k",):
            x = _exact_turn(s[name], s) if name == "k" else s[name].double()
            if c["kind"] == "fp4":
                y = _exact_blocks(x, s[name + "_scale"].double())
                y[s["slots"] < 0] = 0.0
                out[name] = y
                continue
            shape = (s[name + "_cache"].shape[0], c["h_kv"], c["page"])
            cache = torch.zeros(shape + (c["hd"],), dtype=torch.float64, device="cuda")
            if c["kind"] == "rows":
                amax = x.abs().amax(-1)
                unit = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
                scales = torch.ones(shape, dtype=torch.float64, device="cuda")
                scales[block, :, off] = unit[live]
                cache[block, :, off] = _exact_e4m3(x / unit[..., None])[live]
                out[name], out[name + "_row_scales"] = cache, scales
            else:
                cache[block, :, off] = _exact_e4m3(x / s[name + "_scale"].double())[live]
                out[name] = cache
        return out
    grid = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    grid = torch.cat((grid, -grid))

    def unpacked(codes, blocks):
        e = torch.empty(codes.shape[:-1] + (c["hd"],), dtype=torch.float64, device="cuda")
        e[..., 0::2] = grid[(codes & 15).long()]
        e[..., 1::2] = grid[(codes >> 4).long()]
        return e * blocks.double().repeat_interleave(16, -1)

    if c["op"] == "read":
        at = s["slots"].long()
        block, off = at // c["page"], at % c["page"]
        if c["kind"] == "fp4":
            return unpacked(s["cache"][block, :, off], s["blocks"].view(torch.uint8)[block, :, off].view(E4M3)) \
                * s["scale"].double()
        codes = s["cache"][block, :, off].view(E4M3).double()
        return codes * (s["row_scales"][block, :, off].double()[..., None] if c["kind"] == "rows" else s["scale"].double())
    lens = s["lens"].tolist()
    heads = c["h_kv"] * c["group"]
    out = torch.zeros((c["bs"], c["q_len"], heads, c["hd"]), dtype=torch.float64, device="cuda")
    lse = torch.full((c["bs"], c["q_len"], heads), -math.inf, dtype=torch.float64, device="cuda")
    for b, keys in enumerate(lens):
        pages = s["table"][b, :-(-keys // c["page"])].long()
        for h in range(c["h_kv"]):
            rows = slice(h * c["group"], (h + 1) * c["group"])
            k, v = (unpacked(s[x + "_cache"][pages, h], s[x + "_blocks"].view(torch.uint8)[pages, h].view(E4M3))
                    .reshape(-1, c["hd"])[:keys] * s[x + "_scale"].double() for x in ("k", "v"))
            for i in range(c["q_len"]):
                start = keys - c["q_len"]
                lo = max(0, start + i - c["window"] + 1) if c["window"] else 0
                see = torch.arange(keys, device="cuda")
                inside = see >= start
                ok = ~inside | (see <= start + i)
                if s["mask"] is not None:
                    allowed = s["mask"][b, i].bool()
                    ok = ~inside | allowed[(see - start).clamp(0, c["q_len"] - 1)]
                ok &= see >= lo
                score = s["q"][b, i, rows].double() @ k.T * s["softmax_scale"]
                score[:, ~ok] = -math.inf
                if s["sinks"] is not None:
                    score = torch.cat((score, s["sinks"][rows].double()[:, None]), 1)
                if score.shape[1] == 0 or (s["sinks"] is None and not bool(ok.any())):
                    continue
                lse[b, i, rows] = torch.logsumexp(score, 1)
                p = torch.softmax(score, 1)[:, :keys]
                out[b, i, rows] = p @ v
    return {"out": out, "lse": lse}
