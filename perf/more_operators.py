"""Cases for operators that read less of the cache in a decoding step, and for filling it in one pass.

append   rotary positions on the queries and keys of new tokens and the keys and values into the pages of a cache, in one call
store    new tokens into a cache of 4-bit floats (a scale for 16 elements, a power of two a row), and the sequences read back
decode   attention of one new token a sequence over such a cache, grouped heads
bounds   the lowest and highest key of every channel in the pages that got new tokens, as 8-bit integers
sparse   the pages whose keys can score highest, by those bounds, and the attention of one new token over them

`run` computes an operator from elementary torch operations in float32 (angles in float64) while `own` is false, and calls the
library's entry points while it is true.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------- cases
def _case(name, op, b, hkv, d, page, longest, dtype, cache, order, **more):
    return {"name": name, "op": op, "b": b, "hkv": hkv, "d": d, "page": page, "longest": longest, "dtype": dtype, "cache": cache,
            "order": order, **more}


def listed():
    return [
        # one decoding step's queries and keys turned, and the new rows into an 8-bit cache
        _case("append step e4m3", "append", 33, 8, 128, 16, 4096, "bf16", "e4m3", "hnd", new=1, group=4, rot=128, pairs="half"),
        # prompts of several requests into a 16-bit cache, token-major pages
        _case("append prompts 16-bit", "append", 6, 8, 128, 64, 6100, "bf16", "same", "nhd", new=0, group=4, rot=128, pairs="half"),
        # many long prompts into an 8-bit cache, half of each head turned
        _case("append prompts e4m3", "append", 11, 16, 64, 32, 16384, "f16", "e4m3", "hnd", new=0, group=1, rot=32, pairs="interleaved"),
        # a step of a few requests with short contexts, and their cache read back
        _case("store step", "store", 5, 4, 128, 16, 777, "bf16", "e2m1", "hnd", new=1, group=2, rot=128, pairs="half"),
        # prompts that came with their keys turned, stored and read back for their next part's attention
        _case("store prompts", "store", 9, 8, 128, 16, 16384, "bf16", "e2m1", "nhd", new=0, group=4, rot=0, pairs="half"),
        # one sequence: the latency of a step
        _case("decode one", "decode", 1, 8, 128, 16, 1000, "bf16", "e2m1", "hnd", group=4, window=0),
        # a serving batch
        _case("decode batch", "decode", 32, 8, 128, 16, 8192, "bf16", "e2m1", "hnd", group=8, window=0),
        # long contexts, token-major pages
        _case("decode long", "decode", 21, 8, 64, 64, 65536, "f16", "e2m1", "nhd", group=8, window=0),
        # the pages that a step's new tokens lie in
        _case("bounds step", "bounds", 33, 8, 128, 16, 4096, "bf16", "same", "hnd", new=1),
        # the pages of prompts
        _case("bounds prompts", "bounds", 9, 8, 128, 32, 16384, "bf16", "e4m3", "nhd", new=0),
        # one long sequence, 2048 of its keys
        _case("sparse one", "sparse", 1, 8, 128, 16, 30011, "bf16", "same", "hnd", group=4, budget=128, first=1, recent=2),
        # a serving batch of long contexts in 4 bits, 2048 keys of each
        _case("sparse batch", "sparse", 16, 8, 128, 32, 65536, "bf16", "e2m1", "hnd", group=8, budget=64, first=1, recent=2),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "store", "decode", "decode", "bounds", "sparse", "sparse"])
    dtype, order = rng.choice(["bf16", "f16"]), rng.choice(["hnd", "nhd"])
    cache = "e2m1" if op in ("store", "decode") else rng.choice(["same", "e4m3"] if op == "append" else ["same", "e4m3", "e2m1"])
    b, hkv, d = _spread(rng, 1, 40), rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([32, 64, 96, 128] if cache == "e2m1" else [32, 64, 80, 96, 128])
    page = rng.choice([8, 16, 24, 32, 64, 128] if op == "sparse" else [1, 8, 16, 24, 32, 64, 128])
    group = rng.choice([1, 2, 3, 4, 8] if op in ("append", "store") else [1, 2, 3, 4, 8, 16, 20])
    room = {"append": (1 << 28) // (group + 2), "store": 1 << 26, "decode": 1 << 28, "bounds": 1 << 26, "sparse": 1 << 28}[op] // (b * hkv * d)
    longest = _spread(rng, 1, max(2, min(131072, room)))
    more = {}
    if op in ("append", "store"):
        more = {"new": rng.choice([0, 1]), "group": group, "rot": rng.choice([d, d, 32, 16]),
                "pairs": rng.choice(["half", "interleaved"])}
        if op == "store" and (more["new"] == 0 or b * hkv * d > 1 << 15):
            more["rot"] = 0
    if op == "bounds":
        more = {"new": rng.choice([0, 1])}
    if op == "decode":
        more = {"group": group, "window": rng.choice([0, 0, 0, _spread(rng, 1, max(2, longest))])}
    if op == "sparse":
        first, recent = rng.choice([0, 1, 2]), rng.choice([0, 1, 2, 3])
        more = {"group": group, "first": first, "recent": recent,
                "budget": max(1, first + recent, _spread(rng, 4, max(5, min(256, 4096 // page))))}
    return {k: v for k, v in _case("", op, b, hkv, d, page, longest, dtype, cache, order, **more).items() if k != "name"}


def _lens(case):
    """The sequences' lengths: the longest one first, the others spread down to a quarter of it; an empty and a one-token one in a batch."""
    rng = random.Random(1000003 * case["b"] + case["longest"])
    lens = [case["longest"]] + [rng.randint(max(1, case["longest"] // 4), case["longest"]) for _ in range(case["b"] - 1)]
    if case["b"] >= 5:
        lens[2] = 1
        if "new" not in case:
            lens[3] = 0
    return lens


def _fresh(case, lens):
    """New tokens of each sequence: one, or its last three quarters or so (a prompt behind a shared beginning)."""
    return [1] * len(lens) if case["new"] == 1 else [n - n // 4 for n in lens]


def _touched(case, lens):
    """How many pages got new tokens."""
    return sum((n - 1) // case["page"] - (n - f) // case["page"] + 1 for n, f in zip(lens, _fresh(case, lens)))


# ---------------------------------------------------------------------------- 8-bit and 4-bit rows
def _exp8(a):
    """The e4m3 row's exponent: the smallest with a <= 448 * 2^e, no less than -60; 0 for a row of zeros."""
    m, k = torch.frexp(a)
    return torch.where(a == 0, torch.zeros_like(k), k - 9 + (m > 0.875)).clamp(-60, 127)


def _exp4(a):
    """The 4-bit row's exponent: a < 1024 * 2^e, no less than -60; 0 for a row of zeros."""
    k = torch.frexp(a)[1]
    return torch.where(a == 0, torch.zeros_like(k), (k - 10).clamp(-60, 120))


def _codes8(x, e):
    return torch.ldexp(x, -e[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _codes4(x, e):
    """The packed codes (the even element in the low four bits) and the groups' scales of float32 rows."""
    y = torch.ldexp(x, -e[..., None]).unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1) / 6).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    z = torch.where(s == 0, torch.zeros_like(y), y.abs() / torch.where(s == 0, torch.ones_like(s), s))
    # nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; in the middle the even code
    c = (z > 0.25).int() + (z >= 0.75) + (z > 1.25) + (z >= 1.75) + (z > 2.5) + (z >= 3.5) + (z > 5)
    c = (c + 8 * torch.signbit(y)).flatten(-2)
    return (c[..., ::2] + 16 * c[..., 1::2]).to(torch.uint8), scale


def _values4(packed, scale, byte):
    """What 4-bit rows stand for, in float32."""
    of = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=packed.device)
    of = torch.cat([of, -of])
    c = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).int()
    x = of[c].unflatten(-1, (-1, 16)) * scale.float()[..., None]
    return torch.ldexp(x.flatten(-2), byte.int()[..., None] - 127)


# ---------------------------------------------------------------------------- inputs
def _values(gen, shape, dtype, d):
    """Rows as projections give them: unit values with a few channels several times as large."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    lift = torch.ones(d, device="cuda", dtype=dtype)
    lift[torch.randperm(d, generator=gen, device="cuda")[: max(1, d // 32)]] = 4.0
    return x.mul_(lift)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    s = dict(case)
    dt, lens = _TYPES[case["dtype"]], _lens(case)
    b, hkv, d, page = case["b"], case["hkv"], case["d"], case["page"]
    wide = -(-max(lens) // page)
    pages = sum(-(-n // page) for n in lens) + 3
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).cpu()
    table, at = torch.zeros(b, wide, dtype=torch.int32), 0
    for i, n in enumerate(lens):
        table[i, : -(-n // page)] = perm[at: at - (-n // page)]
        at += -(-n // page)
    s["table"], s["lens"] = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    shape = (pages, hkv, page, d) if case["order"] == "hnd" else (pages, page, hkv, d)
    hnd = (lambda t: t) if case["order"] == "hnd" else (lambda t: t.transpose(1, 2))
    for side in ("k", "v"):
        s[side + "_exp"] = s[side + "_scale"] = None
        rows = _values(gen, shape, dt, d)
        if case["cache"] == "e4m3":
            rows = rows.float()
            e = _exp8(rows.abs().amax(-1))
            s[side + "_exp"] = hnd((e + 127).to(torch.uint8)).contiguous()
            rows = _codes8(rows, e)
        elif case["cache"] == "e2m1":
            parts = []
            for part in rows.split(max(1, (1 << 26) // rows[0].numel())):
                part = part.float()
                e = _exp4(part.abs().amax(-1))
                codes, scale = _codes4(part, e)
                parts.append((codes, scale.view(torch.uint8), (e + 127).to(torch.uint8)))
            rows, scale, e = (torch.cat(x) for x in zip(*parts))
            s[side + "_scale"], s[side + "_exp"] = hnd(scale).contiguous().view(torch.float8_e4m3fn), hnd(e).contiguous()
        s[side + "_pages"] = hnd(rows)
    if "new" in case:
        cu = [0]
        for n in _fresh(case, lens):
            cu.append(cu[-1] + n)
        s["tokens"] = cu[-1]
        s["cu_new"] = None if case["new"] == 1 else torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["op"] in ("append", "store"):
        # queries, keys and values are slices of one projection's output
        hq = hkv * case["group"]
        qkv = _values(gen, (s["tokens"], hq + 2 * hkv, d), dt, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.empty(s["tokens"], hq, d, device="cuda", dtype=dt)
        if case["rot"]:
            i = torch.arange(case["rot"] // 2, dtype=torch.float64)
            s["inv_freq"] = (10000.0 ** (-2.0 * i / case["rot"]) / max(1.0, max(lens) / 8192.0)).cuda()
        s["magnitude"] = 1.0 + 0.1 * math.log(max(1.0, max(lens) / 8192.0))
        if case["op"] == "store":
            s["k_out"], s["v_out"] = (torch.zeros(b, hkv, max(lens), d, device="cuda", dtype=dt) for _ in range(2))
    if case["op"] == "bounds":
        s["bounds"] = torch.zeros(pages, hkv, 2, d, device="cuda", dtype=torch.int8)
        s["bounds_exp"] = torch.full((pages, hkv), 127, device="cuda", dtype=torch.uint8)
    if case["op"] in ("decode", "sparse"):
        hq = hkv * case["group"]
        s["q"] = _values(gen, (b, hq, d), dt, d)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(b, hq, device="cuda", dtype=torch.float32)
        s["workspace"] = torch.empty(32 << 20, device="cuda", dtype=torch.uint8)
    if case["op"] == "sparse":
        live = torch.zeros(pages, dtype=torch.int64, device="cuda")  # keys in each page
        start = torch.arange(wide, device="cuda") * page
        n = (s["lens"][:, None] - start).clamp(0, page).long()
        live.index_put_((s["table"].long()[n > 0],), n[n > 0])
        out = [_bounds_of(s, ids, live[ids]) for ids in torch.arange(pages, device="cuda").split(max(1, (1 << 26) // (hkv * page * d)))]
        s["bounds"], s["bounds_exp"] = (torch.cat(x) for x in zip(*out))
        s["select"] = torch.empty(64 << 20, device="cuda", dtype=torch.uint8)
        s["sel_table"] = torch.empty(b, hkv, case["budget"], device="cuda", dtype=torch.int32)
        s["sel_lens"] = torch.empty(b, hkv, device="cuda", dtype=torch.int32)
    return s


# ---------------------------------------------------------------------------- the plain forms
def _tokens(s):
    """Sequence and position of each new token."""
    if s["cu_new"] is None:
        return torch.arange(s["b"], device="cuda"), s["lens"].long() - 1
    cu = s["cu_new"].long()
    t = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True)
    return seq, s["lens"].long()[seq] - cu[seq + 1] + t


def _rotate(s, x, pos):
    """[T, H, D] rows in float32."""
    x, r = x.float(), s["rot"] // 2
    if r == 0:
        return x
    angle = (pos.double()[:, None] * s["inv_freq"])[:, None]
    cos, sin = (angle.cos() * s["magnitude"]).float(), (angle.sin() * s["magnitude"]).float()
    if s["pairs"] == "half":
        x1, x2 = x[..., :r], x[..., r:2 * r]
        return torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin, x[..., 2 * r:]], -1)
    x1, x2 = x[..., :2 * r:2], x[..., 1:2 * r:2]
    return torch.cat([torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2), x[..., 2 * r:]], -1)


def _append(s):
    seq, pos = _tokens(s)
    page, slot = s["table"].long()[seq, pos // s["page"]], pos % s["page"]
    if s["rot"]:
        s["q_out"].copy_(_rotate(s, s["q"], pos).to(s["q"].dtype))
    grow = max(0, math.ceil(math.log2(s["magnitude"])))
    for side, turns in (("k", s["rot"] > 0), ("v", False)):
        x = s[side].float()
        a = x.abs().amax(-1)
        if turns:
            x = _rotate(s, s[side], pos)
        if s["cache"] == "same":
            s[side + "_pages"][page, :, slot] = x.to(s[side].dtype)
            continue
        # the exponent of the row before its rotation, with room for what that can add
        if s["cache"] == "e4m3":
            e = _exp8(a) + (1 + grow if turns else 0)
            s[side + "_pages"].view(torch.uint8)[page, :, slot] = _codes8(x, e).view(torch.uint8)
        else:
            e = _exp4(a) + (grow if turns else 0)
            s[side + "_pages"][page, :, slot], scale = _codes4(x, e)
            s[side + "_scale"].view(torch.uint8)[page, :, slot] = scale.view(torch.uint8)
        s[side + "_exp"][page, :, slot] = (e + 127).to(torch.uint8)


def _pages(s, side, ids, heads=None):
    """Pages `ids` (of one head each with `heads`) as float32 rows [..., page, d]."""
    pool = s[side + "_pages"]
    at = (ids,) if heads is None else (ids, heads)
    if s["cache"] == "same":
        return pool[at].float()
    exps = s[side + "_exp"][at]
    if s["cache"] == "e4m3":
        return torch.ldexp(pool.view(torch.uint8)[at].view(torch.float8_e4m3fn).float(), exps.int()[..., None] - 127)
    return _values4(pool[at], s[side + "_scale"].view(torch.uint8)[at].view(torch.float8_e4m3fn), exps)


def _gather(s, side):
    """[B, H, N, D] float32 rows of the sequences' pages."""
    x = _pages(s, side, s["table"].long())
    return x.transpose(1, 2).flatten(2, 3)


def _read(s):
    n = s["k_out"].shape[2]
    live = (torch.arange(n, device="cuda") < s["lens"][:, None])[:, None, :, None]
    for side in ("k", "v"):
        out = s[side + "_out"]
        out.copy_(torch.where(live, _gather(s, side)[:, :, :n].to(out.dtype), out))


def _attention(s, k, v, live):
    """q over rows [B, H, N, D], of which `live` count."""
    live = live[:, :, None, :]
    q = s["q"].float().unflatten(1, (s["hkv"], s["group"]))
    score = (q @ k.transpose(-1, -2)) / math.sqrt(s["d"])
    score = score.masked_fill(~live, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ v.masked_fill(~live.transpose(-1, -2), 0.0)) / torch.where(total == 0, torch.ones_like(total), total)
    return o.flatten(1, 2).to(s["q"].dtype), (top + total.log())[..., 0].flatten(1, 2)


def _attend(s):
    k, v = (_gather(s, c) for c in ("k", "v"))
    at, lens = torch.arange(k.shape[2], device="cuda"), s["lens"][:, None]
    live = at < lens
    if s["window"]:
        live = live & (at >= lens - s["window"])
    return _attention(s, k, v, live[:, None])


def _bounds_of(s, ids, live):
    """Bounds and their exponents of pages `ids`, of which the first `live` keys count."""
    k = _pages(s, "k", ids)
    on = (torch.arange(s["page"], device="cuda") < live[:, None])[:, None, :, None]
    hi = k.masked_fill(~on, -math.inf).amax(2)
    lo = k.masked_fill(~on, math.inf).amin(2)
    none = (live == 0)[:, None, None]
    hi, lo = hi.masked_fill(none, 0.0), lo.masked_fill(none, 0.0)
    a = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    m, n = torch.frexp(a)
    e = torch.where(a == 0, torch.zeros_like(n), n - 7 + (m > 127 / 128)).clamp(-60, 127)
    codes = torch.stack([torch.ldexp(lo, -e[..., None]).floor(), torch.ldexp(hi, -e[..., None]).ceil()], 2)
    return codes.to(torch.int8), (e + 127).to(torch.uint8)


def _bounds(s):
    lens = s["lens"].long()
    new = torch.ones_like(lens) if s["cu_new"] is None else s["cu_new"].long().diff()
    first, last = (lens - new) // s["page"], (lens - 1) // s["page"]
    ends = (last - first + 1).cumsum(0)
    t = torch.arange(_touched(s, _lens(s)), device="cuda")
    seq = torch.searchsorted(ends, t, right=True)
    j = last[seq] + 1 + t - ends[seq]
    ids = s["table"].long()[seq, j]
    s["bounds"][ids], s["bounds_exp"][ids] = _bounds_of(s, ids, (lens[seq] - j * s["page"]).clamp(max=s["page"]))


def _select(s):
    lens, page, budget = s["lens"].long(), s["page"], s["budget"]
    wide = s["table"].shape[1]
    count = (lens + page - 1) // page
    j = torch.arange(wide, device="cuda")
    ids = torch.where(j < count[:, None], s["table"].long(), torch.zeros_like(s["table"]))
    q = s["q"].float().unflatten(1, (s["hkv"], s["group"]))
    a = q.abs().amax(-1)
    m, n = torch.frexp(a)
    e = torch.where(a == 0, torch.zeros_like(n), n - 7 + (m > 127 / 128)).clamp(-60, 127)
    q = torch.ldexp(q, -e[..., None]).round()
    lo, hi = s["bounds"][ids].permute(3, 0, 2, 4, 1).float()  # [B, H, D, W] each; the sums are integers below 2^24
    u = q.clamp(min=0) @ hi + q.clamp(max=0) @ lo
    score = torch.ldexp(torch.ldexp(u, e[..., None]).amax(2), s["bounds_exp"][ids].transpose(1, 2).int() - 127)
    forced = (j < s["first"]) | (j >= count[:, None] - s["recent"])
    score = torch.where(forced[:, None], torch.full_like(score, math.inf), score)
    score = torch.where((j < count[:, None])[:, None], score, torch.full_like(score, -math.inf))
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    taken = torch.where(order < count[:, None, None], order, wide).sort(-1).values
    if wide < budget:
        taken = torch.cat([taken, torch.full((*taken.shape[:2], budget - wide), wide, device="cuda")], -1)
    real = taken < wide
    pages = ids[:, None].expand(-1, s["hkv"], -1).gather(2, taken.clamp(max=wide - 1))
    short = (taken == count[:, None, None] - 1).any(-1) * (count * page - lens)[:, None]
    s["sel_table"].copy_(torch.where(real, pages, -1))
    s["sel_lens"].copy_(real.sum(-1) * page - short)


def _sparse(s):
    _select(s)
    heads = torch.arange(s["hkv"], device="cuda")[:, None]
    k, v = (_pages(s, c, s["sel_table"].long().clamp(min=0), heads).flatten(2, 3) for c in ("k", "v"))
    live = torch.arange(k.shape[2], device="cuda") < s["sel_lens"][..., None]
    return _attention(s, k, v, live)


# ---------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    if s["op"] == "append":
        _append(s)
        return _stored(s)
    if s["op"] == "store":
        _append(s)
        _read(s)
        return _read_back(s)
    if s["op"] == "decode":
        return _attend(s)
    if s["op"] == "bounds":
        _bounds(s)
        return s["bounds"], s["bounds_exp"]
    return (*_sparse(s), s["sel_table"], s["sel_lens"])


def _stored(s):
    return {c: s[c] for c in ("k_pages", "v_pages", "k_exp", "v_exp", "q_out") if s[c] is not None}


def _read_back(s):
    return {c: s[c] for c in ("k_out", "v_out", "q_out") if c != "q_out" or s["rot"]}


def _own(s):
    from attention_fa2_forward_02_gb300 import binding as fa2
    scales = {c: s[c] for c in ("k_exp", "v_exp", "k_scale", "v_scale")}
    pools = s["k_pages"], s["v_pages"]
    if s["op"] in ("append", "store"):
        if s["rot"]:
            fa2.fa2_rope_append(*pools, s["k"], s["v"], s["inv_freq"], s["table"], s["lens"], q=s["q"], q_out=s["q_out"],
                                cu_new=s["cu_new"], interleaved=s["pairs"] == "interleaved", magnitude=s["magnitude"], **scales)
        else:
            fa2.fa2_kv_append(*pools, s["k"], s["v"], s["table"], s["lens"], cu_new=s["cu_new"], **scales)
        if s["op"] == "append":
            return _stored(s)
        fa2.fa2_kv_read(*pools, s["k_out"], s["v_out"], s["table"], s["lens"], **scales)
        return _read_back(s)
    if s["op"] == "decode":
        fa2.fa2_decode(s["q"], *pools, s["o"], s["lse"], s["table"], s["lens"], s["workspace"], 1 / math.sqrt(s["d"]),
                       window=s["window"], **scales)
        return s["o"], s["lse"]
    if s["op"] == "bounds":
        fa2.fa2_kv_bounds(s["k_pages"], s["bounds"], s["bounds_exp"], s["table"], s["lens"], s["tokens"], cu_new=s["cu_new"],
                          k_exp=s["k_exp"], k_scale=s["k_scale"])
        return s["bounds"], s["bounds_exp"]
    fa2.fa2_select_pages(s["q"], s["bounds"], s["bounds_exp"], s["table"], s["lens"], s["sel_table"], s["sel_lens"], s["select"],
                         s["page"], first=s["first"], recent=s["recent"])
    fa2.fa2_decode_selected(s["q"], *pools, s["o"], s["lse"], s["sel_table"], s["sel_lens"], s["workspace"], 1 / math.sqrt(s["d"]),
                            **scales)
    return s["o"], s["lse"], s["sel_table"], s["sel_lens"]


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    lens, size = _lens(case), 2
    row = case["hkv"] * case["d"]  # elements of a token's keys
    held = {"same": 2 * row, "e4m3": row + case["hkv"], "e2m1": row // 2 + row // 16 + case["hkv"]}[case["cache"]]
    q = row * case.get("group", 0)
    if case["op"] in ("append", "store"):
        n, turned = sum(_fresh(case, lens)), case["rot"] > 0
        w = {"bytes": n * (2 * (row * size + held) + turned * 2 * q * size), "flops": n * (turned * 3 * (row + q) * case["rot"] // case["d"] + 4 * row)}
        if case["op"] == "store":
            n = sum(lens)
            w = {"bytes": w["bytes"] + 2 * n * (row * size + held), "flops": w["flops"] + 4 * n * row}
        return w
    if case["op"] == "bounds":
        fresh = _fresh(case, lens)
        n = sum(a - (a - f) // case["page"] * case["page"] for a, f in zip(lens, fresh))  # keys of the pages touched
        return {"bytes": n * held + _touched(case, lens) * (2 * row + case["hkv"]), "flops": 2 * n * row}
    if case["op"] == "decode":
        n = sum(min(x, case["window"]) if case["window"] else x for x in lens)
        w = {"bytes": 2 * n * held, "flops": 4 * n * q}
    else:
        n = sum(min(x, case["budget"] * case["page"]) for x in lens)
        pages = sum(-(-x // case["page"]) for x in lens)
        w = {"bytes": 2 * n * held + pages * (2 * row + case["hkv"]) + case["b"] * case["hkv"] * (case["budget"] + 1) * 4,
             "flops": 4 * n * q + 2 * pages * q}
    return {"bytes": w["bytes"] + case["b"] * q * (2 * size) + case["b"] * q // case["d"] * 4, "flops": w["flops"]}


# ---------------------------------------------------------------------------- the definitions in 64 bits
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e4m3_64(codes):
    """What e4m3 bytes stand for, from their bits: sign, 4 exponent bits (bias 7), 3 fraction bits; all ones is NaN."""
    c = codes.view(torch.uint8).to(torch.int64)
    e, f = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2((e - 7).double()))
    mag = torch.where((c & 127) == 127, torch.full_like(mag, math.nan), mag)
    return torch.where(c >= 128, -mag, mag)


def _rows64(s, side, ids):
    """Rows of pages `ids` in 64 bits."""
    pool = s[side + "_pages"]
    if s["cache"] == "same":
        return pool[ids].double()
    two = torch.exp2(s[side + "_exp"][ids].double() - 127)[..., None]
    if s["cache"] == "e4m3":
        return _e4m3_64(pool.view(torch.uint8)[ids]) * two
    codes = pool[ids].to(torch.int64)
    codes = torch.stack([codes % 16, codes // 16], -1).flatten(-2)
    value = torch.tensor(_E2M1 + [-x for x in _E2M1], dtype=torch.float64, device="cuda")[codes]
    return value * _e4m3_64(s[side + "_scale"].view(torch.uint8)[ids]).repeat_interleave(16, -1) * two


def _nearest_e4m3_64(y):
    """The e4m3 value nearest to each element, ties to the even fraction."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _nearest_e2m1_64(y):
    """The 4-bit value nearest to each element, ties to the even code."""
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0)).double()
    return (torch.round(y / step) * step).clamp(-6, 6)


def _turned64(s, x, pos):
    y, r = x.double(), s["rot"] // 2
    if r == 0:
        return y
    turn = (torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, None] * s["inv_freq"]) * s["magnitude"])[:, None]
    y = y.clone()
    one, two = (slice(0, r), slice(r, 2 * r)) if s["pairs"] == "half" else (slice(0, 2 * r, 2), slice(1, 2 * r, 2))
    z = torch.complex(y[..., one], y[..., two]) * turn
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _log2_floor(a):
    """floor(log2(a)) of positive numbers."""
    e = torch.floor(torch.log2(a))
    e = torch.where(torch.exp2(e) > a, e - 1, e)
    return torch.where(torch.exp2(e + 1) <= a, e + 1, e)


def _smallest64(a, most):
    """The smallest e with a <= most * 2^e, no less than -60; 0 for 0."""
    e = torch.ceil(torch.log2(a.clamp(min=1e-300) / most))
    e = torch.where(a <= most * torch.exp2(e - 1), e - 1, e)
    e = torch.where(a > most * torch.exp2(e), e + 1, e)
    return torch.where(a > 0, e.clamp(min=-60), torch.zeros_like(e))


def exact(case, seed):
    s = prepare(case, seed)
    lens, b, hkv, d, page = _lens(case), case["b"], case["hkv"], case["d"], case["page"]
    table = s["table"].long()
    if case["op"] in ("append", "store"):
        fresh, at, out, kept = _fresh(case, lens), 0, {}, {}
        pos = torch.cat([torch.arange(n - f, n, device="cuda") for n, f in zip(lens, fresh)])
        ids = torch.cat([table[i][torch.arange(n - f, n, device="cuda") // page] for i, (n, f) in enumerate(zip(lens, fresh))])
        add = math.ceil(math.log2(s["magnitude"])) if s["magnitude"] > 1 else 0
        if case["op"] == "append":
            for side in ("k", "v"):
                turns = side == "k" and case["rot"] > 0
                rows = _turned64(s, s[side], pos) if turns else s[side].double()
                pool = _e4m3_64(s[side + "_pages"]) if case["cache"] == "e4m3" else s[side + "_pages"].double()
                if case["cache"] == "e4m3":
                    e = _smallest64(s[side].double().abs().amax(-1), 448.0) + (1 + add if turns else 0)
                    rows = _nearest_e4m3_64(rows * torch.exp2(-e)[..., None])
                    out[side + "_exp"] = s[side + "_exp"].clone()
                    out[side + "_exp"][ids, :, pos % page] = (e + 127).to(torch.uint8)
                pool[ids, :, pos % page] = rows
                out[side + "_pages"] = pool
        else:
            for side in ("k", "v"):
                full = torch.zeros(b, hkv, max(lens), d, dtype=torch.float64, device="cuda")
                for i, (n, f) in enumerate(zip(lens, fresh)):
                    full[i, :, :n] = _rows64(s, side, table[i, : -(-n // page)]).transpose(0, 1).flatten(1, 2)[:, :n]
                    x = s[side][at: at + f].double()
                    a = x.abs().amax(-1)
                    e = torch.where(a > 0, (_log2_floor(a.clamp(min=1e-300)) - 9).clamp(min=-60), torch.zeros_like(a))
                    if side == "k" and case["rot"]:
                        x, e = _turned64(s, s[side][at: at + f], pos[at: at + f]), e + add
                    y = (x * torch.exp2(-e)[..., None]).unflatten(-1, (-1, 16))
                    g = _nearest_e4m3_64(y.abs().amax(-1, keepdim=True) / 6)
                    y = torch.where(g > 0, _nearest_e2m1_64(y / g.clamp(min=1e-300)) * g, torch.zeros_like(y)).flatten(-2)
                    full[i, :, n - f:n] = (y * torch.exp2(e)[..., None]).transpose(0, 1)
                    at += f
                at = 0
                out[side + "_out"] = full
        if case["rot"] or case["op"] == "append":
            out["q_out"] = _turned64(s, s["q"], pos)
        return out
    if case["op"] == "bounds":
        codes, exps = s["bounds"].clone(), s["bounds_exp"].clone()
        for i, (n, f) in enumerate(zip(lens, _fresh(case, lens))):
            j = torch.arange((n - f) // page, (n - 1) // page + 1, device="cuda")
            k = _rows64(s, "k", table[i, j])
            tail = n - int(j[-1]) * page
            low, high = k.clone(), k
            low[-1, :, tail:], high[-1, :, tail:] = math.inf, -math.inf
            low, high = low.amin(2), high.amax(2)
            e = _smallest64(torch.maximum(low.abs(), high.abs()).amax(-1), 127.0)
            codes[table[i, j]] = torch.stack([torch.floor(low * torch.exp2(-e)[..., None]), torch.ceil(high * torch.exp2(-e)[..., None])], 2).to(torch.int8)
            exps[table[i, j]] = (e + 127).to(torch.uint8)
        return codes, exps
    hq, group = hkv * case["group"], case["group"]
    o = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    if case["op"] == "sparse":
        sel, sel_lens = torch.full_like(s["sel_table"], -1), torch.zeros_like(s["sel_lens"])
    for i, n in enumerate(lens):
        first = max(0, n - case["window"]) if case.get("window") else 0
        if n - first <= 0:
            continue
        q = s["q"][i].double().view(hkv, group, d)
        used = -(-n // page)
        if case["op"] == "sparse":
            e = _smallest64(q.abs().amax(-1), 127.0)
            codes = torch.round(q * torch.exp2(-e)[..., None])[None]                       # [1, H, G, D]
            lo, hi = s["bounds"][table[i, :used]].double().unbind(2)                      # [W, H, D] each
            score = torch.empty(used, hkv, dtype=torch.float64, device="cuda")
            for part in torch.arange(used, device="cuda").split(max(1, (1 << 25) // (hq * d))):
                u = torch.maximum(codes * lo[part][:, :, None], codes * hi[part][:, :, None]).sum(-1)
                score[part] = (u * torch.exp2(e)).amax(-1) * torch.exp2(s["bounds_exp"][table[i, part]].double() - 127)
            score[: case["first"]] = math.inf
            score[max(0, used - case["recent"]):] = math.inf
            for h in range(hkv):
                # the largest ones, the earlier of two alike: every score's rank by counting
                top = torch.sort(-score[:, h], stable=True).indices[: case["budget"]].sort().values
                held = top.numel() * page - (used * page - n if int(top[-1]) == used - 1 else 0)
                sel[i, h, : top.numel()], sel_lens[i, h] = table[i, top].int(), held
                k, v = (_rows64(s, c, table[i, top])[:, h].flatten(0, 1)[:held] for c in ("k", "v"))
                rows = slice(h * group, (h + 1) * group)
                x = q[h] @ k.T / math.sqrt(d)
                lse[i, rows], o[i, rows] = torch.logsumexp(x, -1), torch.softmax(x, -1) @ v
            continue
        k, v = (_rows64(s, c, table[i, :used]).transpose(0, 1).flatten(1, 2)[:, first:n] for c in ("k", "v"))
        x = torch.einsum("hgd,hnd->hgn", q, k) / math.sqrt(d)
        lse[i] = torch.logsumexp(x, -1).flatten()
        o[i] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), v).reshape(hq, d)
    return (o, lse, sel, sel_lens) if case["op"] == "sparse" else (o, lse)
