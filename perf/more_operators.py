"""Cases of cross attention, attention to shared prefixes and the merge of partial attention results.

Each case is one pass through one operator.  ``run`` computes it either in
elementary torch operations (``own`` false) or through the library's public
entry points (``own`` true); both take what ``prepare`` makes.  ``exact``
gives the same outputs from the definitions in 64 bits, written apart from
the plain form.

Keys and values lie in paged caches [blocks, KV heads, page, head dim] of
E4M3 codes with one float32 scale each (kind "tensor") or one per cached row
(kind "rows").  Query head h reads KV head h // group.
"""

import math

import torch

own = False

E4M3 = torch.float8_e4m3fn

# ------------------------------------------------------------------ cases --


def listed():
    cross = dict(op="cross", h_kv=8, group=4, hd=128, page=16, kind="tensor", empty=0, pad=0)
    shared = dict(op="shared", h_kv=8, group=4, hd=128, page=16, kind="tensor", q_len=1, mask=False, sinks=False,
                  alone=0)
    merge = dict(op="merge", heads=32, hd=128)
    return [
        # the next token of one sequence, reading its encoder's states: the smallest call, latency
        dict(cross, name="cross one token", bs=1, q_lo=1, q_hi=1, k_lo=777, k_hi=777, h_kv=16, group=1, hd=64),
        # a decode step of 64 sequences, each with states of another length, one of them without any
        dict(cross, name="cross decode step", bs=64, q_lo=1, q_hi=1, k_lo=128, k_hi=1600, kind="rows", empty=1),
        # prompts of eight sequences to states of unlike lengths, one KV head per query head
        dict(cross, name="cross prompts", bs=8, q_lo=5, q_hi=448, k_lo=100, k_hi=1500, h_kv=16, group=1, hd=64,
             page=64, empty=1, pad=9),
        # one long prompt to an image's states in cache rows with a scale each
        dict(cross, name="cross long prompt", bs=1, q_lo=2047, q_hi=2047, k_lo=6404, k_hi=6404, kind="rows", page=32),
        # a prompt chunk to the states of a long document: the matrix products carry it
        dict(cross, name="cross document", bs=1, q_lo=2048, q_hi=2048, k_lo=16384, k_hi=16384, page=64),
        # four answers drawn from one short prompt: latency
        dict(shared, name="shared four samples", bs=4, groups=1, p_lo=515, p_hi=515, o_lo=1, o_hi=64),
        # a served batch behind one long system prompt
        dict(shared, name="shared batch", bs=64, groups=1, p_lo=32768, p_hi=32768, o_lo=17, o_hi=1024),
        # three prompts with their samples, four drafted tokens a step, sinks, some sequences without a shared prompt
        dict(shared, name="shared drafts", bs=48, groups=3, p_lo=4096, p_hi=16384, o_lo=4, o_hi=2048, q_len=4,
             mask=True, sinks=True, alone=5),
        # many sequences, wide groups of heads, a scale per row
        dict(shared, name="shared many", bs=256, groups=2, p_lo=7000, p_hi=8191, o_lo=100, o_hi=1500, h_kv=4, group=8,
             kind="rows", page=32),
        # two results of a decode step put together
        dict(merge, name="merge step", parts=2, n=64),
        # three results of a prompt put together
        dict(merge, name="merge prompt", parts=3, n=8191),
    ]


MOST_FLOPS = 5e11    # of a drawn case
MOST_KEYS = 1 << 20  # of one KV head, all sequences together


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(["cross", "cross", "shared", "shared", "merge"])
    if op == "merge":
        return dict(op=op, parts=rng.randint(2, 4), n=_log(rng, 1, 8191), heads=rng.choice([1, 8, 16, 28, 32, 64]),
                    hd=rng.choice([64, 128, 128, 512]))
    hd = rng.choice([64, 128, 128])
    common = dict(op=op, hd=hd, page=rng.choice([16, 16, 32, 64, 128, 256]), kind=rng.choice(["tensor", "rows"]))
    while op == "cross":
        h_kv, group = rng.choice([(1, 8), (2, 7), (4, 1), (4, 8), (8, 3), (8, 4), (16, 1), (8, 8)])
        bs = _log(rng, 1, 64)
        q_hi = 1 if rng.random() < 0.35 else _log(rng, 2, 2048)
        k_hi = _log(rng, 1, 16384)
        c = dict(common, bs=bs, q_lo=1 if q_hi == 1 else rng.choice([0, 1, q_hi]), q_hi=q_hi,
                 k_lo=rng.choice([0, k_hi // 3, k_hi]), k_hi=k_hi, h_kv=h_kv, group=group,
                 empty=int(bs > 2 and rng.random() < 0.3), pad=rng.choice([0, 0, 3]) if q_hi > 1 else 0)
        if bs * q_hi * k_hi * h_kv * group * hd * 4 <= MOST_FLOPS and bs * k_hi <= MOST_KEYS // 2:
            return c
    while True:
        h_kv, group = rng.choice([(1, 8), (2, 7), (4, 4), (4, 8), (8, 3), (8, 4), (8, 1)])
        bs = _log(rng, 1, 256)
        p_hi, o_hi = _log(rng, 1, 32768), _log(rng, 1, 4096)
        q_len = rng.choice([1, 1, 1, 2, 4, 8])
        groups = rng.randint(1, min(bs, 4))
        c = dict(common, bs=bs, groups=groups, p_lo=rng.choice([p_hi // 2, p_hi]), p_hi=p_hi,
                 o_lo=rng.choice([0, 1, o_hi]), o_hi=o_hi, h_kv=h_kv, group=group, q_len=q_len,
                 mask=q_len > 1 and rng.random() < 0.5, sinks=rng.random() < 0.3,
                 alone=rng.randint(0, (bs - groups) // 4))
        if bs * q_len * (p_hi + o_hi) * h_kv * group * hd * 4 <= MOST_FLOPS / 4 and bs * (p_hi + o_hi) <= 4 * MOST_KEYS:
            return c


# ----------------------------------------------------------------- inputs --


def _lengths(g, n, lo, hi):
    """n lengths between lo and hi, the first of them hi."""
    x = torch.randint(lo, hi + 1, (n,), device="cuda", generator=g)
    x[:1] = hi
    return x


def _spread(g, n, lo, hi):
    """n lengths evenly from lo to hi, in random order: their sum is the same every time."""
    x = torch.tensor([hi - (hi - lo) * i // max(n - 1, 1) for i in range(n)], device="cuda")
    return x[torch.randperm(n, device="cuda", generator=g)]


def _starts(lengths):
    return torch.cat((lengths.new_zeros(1), lengths.cumsum(0))).to(torch.int32)


def _tables(g, c, lengths_of):
    """One pool of pages in random order: a table [n, places] for each list of lengths, and the pages in the pool."""
    page = c["page"]
    blocks_of = [(x + page - 1) // page for x in lengths_of]
    used = int(sum(int(b.sum()) for b in blocks_of))
    perm = torch.randperm(used + 2, device="cuda", generator=g)
    tables, first = [], 0
    for b in blocks_of:
        most = max(1, int(b.max()))
        at = torch.arange(most, device="cuda")
        place = first + (b.cumsum(0) - b)[:, None] + at
        t = perm[place.clamp(max=used + 1)]
        tables.append(torch.where(at < b[:, None], t, torch.zeros_like(t)).to(torch.int32))
        first += int(b.sum())
    return tables, used + 2


def _caches(g, c, blocks):
    """K and V of a projection (normal values, some dimensions several times the others) as codes and scales."""
    s = {}
    for name in ("k", "v"):
        x = torch.randn((blocks, c["h_kv"], c["page"], c["hd"]), device="cuda", generator=g)
        x *= torch.randn(c["hd"], device="cuda", generator=g).mul_(0.4).exp_()
        if c["kind"] == "rows":
            x *= torch.rand((blocks, c["h_kv"], c["page"], 1), device="cuda", generator=g) + 0.5
            scale = x.abs().amax(-1) / 448.0
            codes = (x / scale[..., None]).clamp(-448, 448)
        else:
            scale = (x.abs().amax() / 448.0).reshape(1)
            codes = (x / scale).clamp(-448, 448)
        s[name + "_cache"], s[name + "_scale"] = codes.to(E4M3), scale
        del x, codes
    return s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "merge":
        outs = [torch.randn((c["n"], c["heads"], c["hd"]), device="cuda", generator=g).to(torch.bfloat16)
                for _ in range(c["parts"])]
        lses = [torch.randn((c["n"], c["heads"]), device="cuda", generator=g) * 3 + 6 for _ in range(c["parts"])]
        for i, (o, l) in enumerate(zip(outs, lses)):  # tokens without a key in this part; one without any at all
            none = torch.rand(c["n"], device="cuda", generator=g) < 0.1
            none[-1] = c["n"] > 1
            o[none], l[none] = 0.0, -math.inf
        return dict(c=c, outs=outs, lses=lses)
    heads = c["h_kv"] * c["group"]
    if c["op"] == "cross":
        q_lens, k_lens = _spread(g, c["bs"], c["q_lo"], c["q_hi"]), _lengths(g, c["bs"], c["k_lo"], c["k_hi"])
        if c["empty"]:
            k_lens[c["bs"] // 2] = 0
        (table,), blocks = _tables(g, c, [k_lens])
        starts = _starts(q_lens)
        s = dict(c=c, table=table, starts=starts, k_lens=k_lens.to(torch.int32), **_caches(g, c, blocks))
        n = int(starts[-1]) + c["pad"]
        s["plan"] = (starts.tolist(), k_lens.tolist())  # the lengths as the host knows them
    else:
        alone = c["alone"]  # sequences in front that share nothing
        per = [(c["bs"] - alone) // c["groups"]] * c["groups"]
        per[0] += c["bs"] - alone - sum(per)
        p_lens, o_lens = _lengths(g, c["groups"], c["p_lo"], c["p_hi"]), _lengths(g, c["bs"], c["o_lo"], c["o_hi"])
        (p_table, o_table), blocks = _tables(g, c, [p_lens, o_lens])
        members = torch.tensor(per, device="cuda")
        s = dict(c=c, p_table=p_table, p_lens=p_lens.to(torch.int32), members=_starts(members) + alone,
                 o_table=o_table, o_lens=o_lens.to(torch.int32), **_caches(g, c, blocks))
        of = [-1] * alone + [i for i, m in enumerate(per) for _ in range(m)]
        s["plan"] = (of, p_lens.tolist(), o_lens.tolist())
        n = c["bs"] * c["q_len"]
        s["mask"] = None
        if c["mask"]:  # a tree of drafted tokens: each sees itself and some before it
            m = torch.rand((c["bs"], c["q_len"], c["q_len"]), device="cuda", generator=g) < 0.6
            s["mask"] = (m.tril() | torch.eye(c["q_len"], dtype=torch.bool, device="cuda")).to(torch.uint8)
        s["sinks"] = torch.randn(heads, device="cuda", generator=g) if c["sinks"] else None
    q = torch.randn((n, heads, c["hd"]), device="cuda", generator=g).to(torch.bfloat16)
    s["q"] = q.unflatten(0, (c["bs"], c["q_len"])) if c["op"] == "shared" else q
    s["softmax_scale"] = c["hd"] ** -0.5
    return s


# ------------------------------------------------------------- plain form --


def _plain_rows(s, name, pages, keys):
    """[h_kv, keys, hd] of the cache in 32 bits."""
    x = s[name + "_cache"][pages].float()
    scale = s[name + "_scale"]
    x = x * (scale[pages][..., None] if s["c"]["kind"] == "rows" else scale)
    return x.transpose(0, 1).reshape(s["c"]["h_kv"], -1, s["c"]["hd"])[:, :keys]


def _plain_attend(s, q, k, v, hidden=None, sinks=None):
    """q [n, heads, hd] to k and v [h_kv, keys, hd]; hidden [n, keys] truth values."""
    c = s["c"]
    n, heads = q.shape[:2]
    q = q.float().reshape(n, c["h_kv"], c["group"], -1).transpose(0, 1).reshape(c["h_kv"], n * c["group"], -1)
    score = (q @ k.transpose(1, 2)) * s["softmax_scale"]
    if hidden is not None:
        score = score.masked_fill_(hidden.repeat_interleave(c["group"], 0)[None], -math.inf)
    if sinks is not None:
        sink = sinks.reshape(c["h_kv"], 1, c["group"]).expand(-1, n, -1).reshape(c["h_kv"], -1, 1)
        score = torch.cat((score, sink), 2)
    if score.shape[2] == 0:
        return q.new_zeros((n, heads, c["hd"])), q.new_full((n, heads), -math.inf)
    top = score.amax(2, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(2, keepdim=True)
    o = p[:, :, :k.shape[1]] @ v
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log())[..., 0]
    back = (c["h_kv"], n, c["group"])
    return (o.reshape(*back, -1).transpose(0, 1).reshape(n, heads, -1),
            lse.reshape(back).transpose(0, 1).reshape(n, heads))


def _plain_cross(s):
    c = s["c"]
    starts, k_lens = s["plan"]
    out = torch.zeros_like(s["q"])
    lse = torch.full(s["q"].shape[:2], -math.inf, device="cuda")
    for b, keys in enumerate(k_lens):
        lo, hi = starts[b], starts[b + 1]
        if hi > lo and keys > 0:
            pages = s["table"][b, :-(-keys // c["page"])].long()
            o, l = _plain_attend(s, s["q"][lo:hi], *(_plain_rows(s, x, pages, keys) for x in "kv"))
            out[lo:hi], lse[lo:hi] = o.to(torch.bfloat16), l
    return out, lse


def _plain_shared(s):
    c = s["c"]
    of, p_lens, o_lens = s["plan"]
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:3], device="cuda")
    last, prefix = None, None
    for b, keys in enumerate(o_lens):
        if of[b] != last:
            last = of[b]
            shared = p_lens[last] if last >= 0 else 0
            pages = s["p_table"][max(last, 0), :-(-shared // c["page"])].long()
            prefix = [_plain_rows(s, x, pages, shared) for x in "kv"]
        pages = s["o_table"][b, :-(-keys // c["page"])].long()
        k, v = (torch.cat((p, _plain_rows(s, x, pages, keys)), 1) for p, x in zip(prefix, "kv"))
        hidden = None
        if c["q_len"] > 1:  # the last q_len keys are the block's own tokens
            at = torch.arange(k.shape[1], device="cuda") - (k.shape[1] - c["q_len"])
            own_key = torch.arange(k.shape[1], device="cuda") >= prefix[0].shape[1]
            i = torch.arange(c["q_len"], device="cuda")[:, None]
            if s["mask"] is None:
                see = at <= i
            else:
                see = s["mask"][b].bool()[:, at.clamp(min=0)]
            hidden = (at >= 0) & own_key & ~see
        o, l = _plain_attend(s, s["q"][b], k, v, hidden, s["sinks"])
        out[b], lse[b] = o.to(torch.bfloat16), l
    return out, lse


def _plain_merge(s):
    lse = torch.stack(s["lses"])
    top = lse.amax(0)
    top0 = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = (lse - top0).exp()
    total = w.sum(0)
    o = sum(x.float() * y[..., None] for x, y in zip(s["outs"], w))
    o = torch.where(total[..., None] > 0, o / total[..., None], torch.zeros_like(o))
    return o.to(torch.bfloat16), top0 + total.log()


# -------------------------------------------------------------------- run --


def run(state):
    s = state
    c = s["c"]
    if not own:
        out, lse = {"cross": _plain_cross, "shared": _plain_shared, "merge": _plain_merge}[c["op"]](s)
        return {"out": out, "lse": lse}
    import paged_decode_attention_fp8_gb300 as fm
    if c["op"] == "cross":
        one = c["q_hi"] == 1 and c["q_lo"] == 1 and not c["pad"]  # a token each: no list of starts
        out, lse = fm.paged_cross_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["k_lens"], s["k_scale"],
                                            s["v_scale"], softmax_scale=s["softmax_scale"],
                                            q_starts=None if one else s["starts"])
    elif c["op"] == "shared":
        out, lse = fm.paged_gqa_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["p_table"], s["p_lens"],
                                              s["members"], s["o_table"], s["o_lens"], s["k_scale"], s["v_scale"],
                                              softmax_scale=s["softmax_scale"], spec_mask=s["mask"], sinks=s["sinks"])
    else:
        out, lse = fm.attention_merge(s["outs"], s["lses"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------- work --


def _sum_of(n, lo, hi):
    """Expected sum of n lengths as _lengths makes them."""
    return hi + (n - 1) * (lo + hi) / 2


def work(case):
    c = case
    if c["op"] == "merge":
        rows = c["n"] * c["heads"]
        return {"bytes": rows * (c["parts"] + 1) * (2 * c["hd"] + 4), "flops": rows * c["parts"] * 2 * c["hd"]}
    heads = c["h_kv"] * c["group"]
    key = c["h_kv"] * 2 * (c["hd"] + (4 if c["kind"] == "rows" else 0))  # bytes of a key and its value
    row = heads * (4 * c["hd"] + 4)                                      # of a token's queries, outputs and sums
    pair = heads * c["hd"] * 4                                           # operations of a token and a key
    if c["op"] == "cross":
        tokens = c["q_hi"] if c["bs"] == 1 else c["bs"] * (c["q_lo"] + c["q_hi"]) / 2
        keys = _sum_of(c["bs"], c["k_lo"], c["k_hi"])
        if c["empty"]:
            keys -= (c["k_lo"] + c["k_hi"]) / 2
        return {"bytes": keys * key + (tokens + c["pad"]) * row, "flops": tokens * keys / c["bs"] * pair}
    tokens = c["bs"] * c["q_len"]
    shared, alone = _sum_of(c["groups"], c["p_lo"], c["p_hi"]), _sum_of(c["bs"], c["o_lo"], c["o_hi"])
    return {"bytes": (shared + alone) * key + tokens * row,
            "flops": (tokens - c["alone"] * c["q_len"]) * shared / c["groups"] * pair + c["q_len"] * alone * pair}


# ---------------------------------------------------- definition, 64 bits --


def _exact_codes(x):
    """E4M3 bytes as the numbers they stand for, from their bits."""
    b = x.view(torch.uint8).long()
    e, m = (b >> 3) & 15, b & 7
    mag = torch.where(e == 0, m.double() * 2.0 ** -9, (8 + m).double() * torch.exp2((e - 10).double()))
    return torch.where(b >= 128, -mag, mag)


def _exact_keys(s, name, table, keys, h):
    """[keys, hd] of KV head h."""
    c = s["c"]
    j = torch.arange(keys, device="cuda")
    block, off = table.long()[j // c["page"]], j % c["page"]
    x = _exact_codes(s[name + "_cache"][block, h, off])
    scale = s[name + "_scale"].double()
    return x * (scale[block, h, off][:, None] if c["kind"] == "rows" else scale)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "merge":
        lse = torch.stack([x.double() for x in s["lses"]], -1)
        total = torch.logsumexp(lse, -1)
        share = (lse - total[..., None]).exp().nan_to_num(0.0)
        return {"out": (torch.stack([x.double() for x in s["outs"]], -1) * share[..., None, :]).sum(-1), "lse": total}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    if c["op"] == "cross":
        starts, k_lens = s["plan"]
        for b, keys in enumerate(k_lens):
            tokens = slice(starts[b], starts[b + 1])
            if starts[b] == starts[b + 1] or keys == 0:
                continue
            for h in range(c["h_kv"]):
                k, v = (_exact_keys(s, x, s["table"][b], keys, h) for x in "kv")
                for q in range(h * c["group"], (h + 1) * c["group"]):
                    score = s["q"][tokens, q].double() @ k.T * s["softmax_scale"]
                    lse[tokens, q] = torch.logsumexp(score, 1)
                    out[tokens, q] = (score - lse[tokens, q][:, None]).exp() @ v
        return {"out": out, "lse": lse}
    of, p_lens, o_lens = s["plan"]
    for h in range(c["h_kv"]):
        heads = slice(h * c["group"], (h + 1) * c["group"])
        front = [[_exact_keys(s, x, s["p_table"][i], keys, h) for x in "kv"] for i, keys in enumerate(p_lens)]
        for b, keys in enumerate(o_lens):
            k, v = (_exact_keys(s, x, s["o_table"][b], keys, h) for x in "kv")
            if of[b] >= 0:
                k, v = torch.cat((front[of[b]][0], k)), torch.cat((front[of[b]][1], v))
            score = torch.einsum("ihd,kd->ihk", s["q"][b, :, heads].double(), k) * s["softmax_scale"]
            for i in range(c["q_len"]):  # key x of the block is len - q_len + x: token i sees it by its mask or order
                for x in range(c["q_len"]):
                    sees = bool(s["mask"][b, i, x]) if c["mask"] else x <= i
                    if keys - c["q_len"] + x >= 0 and not sees:
                        score[i, :, len(k) - c["q_len"] + x] = -math.inf
            if c["sinks"]:
                score = torch.cat((score, s["sinks"][heads].double()[None, :, None].expand(c["q_len"], -1, 1)), 2)
            if score.shape[2] == 0:
                continue
            lse[b, :, heads] = torch.logsumexp(score, 2)
            p = (score - lse[b, :, heads][..., None]).exp().nan_to_num(0.0)
            out[b, :, heads] = torch.einsum("ihk,kd->ihd", p[..., :len(k)], v)
    return {"out": out, "lse": lse}
