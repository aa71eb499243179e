"""Cases for the operators of a serving and training step around the attention kernels.

rope     rotary positions on [B, H, N, D] views, forward and backward
append   new keys and values into the pages of a cache, as 16-bit rows or as e4m3 codes with a power-of-two scale a row
read     pages back to contiguous [B, H, N, D] keys and values
decode   attention of one new token a sequence over a paged cache, grouped heads

`run` computes an operator from elementary torch operations in float32 (angles in float64) while `own` is false, and calls the
library's entry points while it is true.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases
def _rope(name, b, h, n, d, rot, pairs, order, dtype, way, far):
    return {"name": name, "op": "rope", "b": b, "h": h, "n": n, "d": d, "rot": rot, "pairs": pairs, "order": order, "dtype": dtype,
            "way": way, "far": far}


def _cache(name, op, b, hkv, d, page, longest, dtype, cache, order, **more):
    return {"name": name, "op": op, "b": b, "hkv": hkv, "d": d, "page": page, "longest": longest, "dtype": dtype, "cache": cache,
            "order": order, **more}


def listed():
    return [
        # the query and key heads of one decoding step for a few sequences, far into long contexts
        _rope("rope step", 1, 40, 7, 128, 128, "half", "bnhd", "bf16", "forward", 1 << 20),
        # the queries of the training attention (B=2 H=16 N=8192 d=128)
        _rope("rope training", 2, 16, 8192, 128, 128, "interleaved", "bhnd", "bf16", "forward", 8192),
        # the gradient of a packed batch's heads of which a part rotates
        _rope("rope gradient, part", 3, 20, 5003, 96, 32, "half", "bnhd", "f16", "backward", 32768),
        # one new token for each of a batch's sequences into an 8-bit cache
        _cache("append step e4m3", "append", 33, 8, 128, 16, 4096, "bf16", "e4m3", "hnd", new=1),
        # prompts of several requests into a 16-bit cache
        _cache("append prompts 16-bit", "append", 6, 8, 128, 64, 6100, "bf16", "same", "nhd", new=0),
        # many long prompts into an 8-bit cache
        _cache("append prompts e4m3", "append", 11, 16, 64, 32, 16384, "f16", "e4m3", "hnd", new=0),
        # a short context read back for a second prompt chunk
        _cache("read short", "read", 1, 4, 64, 16, 777, "f16", "same", "nhd"),
        # a batch of long contexts read back out of an 8-bit cache
        _cache("read long e4m3", "read", 9, 8, 128, 16, 16384, "bf16", "e4m3", "hnd"),
        # one sequence: the latency of a step
        _cache("decode one", "decode", 1, 8, 128, 16, 1000, "bf16", "same", "hnd", group=4, window=0),
        # a small batch with a head of its own for every query head, sliding window
        _cache("decode window", "decode", 7, 12, 64, 32, 2501, "f16", "same", "nhd", group=1, window=1024),
        # a serving batch over an 8-bit cache
        _cache("decode batch e4m3", "decode", 32, 8, 128, 16, 8192, "bf16", "e4m3", "hnd", group=8, window=0),
        # long contexts
        _cache("decode long", "decode", 21, 8, 128, 64, 65536, "bf16", "same", "nhd", group=8, window=0),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "decode", "decode"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "rope":
        d = rng.choice([32, 64, 80, 96, 128])
        rot = rng.choice([d, d, d // 2, 32, 18])
        h, b = _spread(rng, 1, 64), rng.randint(1, 4)
        n = _spread(rng, 1, max(1, (1 << 25) // (b * h * d)))
        return {k: v for k, v in _rope("", b, h, n, d, rot, rng.choice(["half", "interleaved"]), rng.choice(["bhnd", "bnhd"]),
                                       rng.choice(["bf16", "f16", "f32"]), rng.choice(["forward", "backward"]), _spread(rng, 64, 1 << 20)).items()
                if k != "name"}
    b, hkv, d = _spread(rng, 1, 40), rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([32, 64, 80, 96, 128])
    page, cache, order = rng.choice([1, 8, 16, 24, 32, 64, 128]), rng.choice(["same", "e4m3"]), rng.choice(["hnd", "nhd"])
    room = {"append": 1 << 26, "read": 1 << 26, "decode": 1 << 29}[op] // (b * hkv * d)
    longest = _spread(rng, 1, max(2, min(131072, room)))
    more = {}
    if op == "append":
        more["new"] = rng.choice([0, 1])
    if op == "decode":
        more["group"] = rng.choice([1, 2, 3, 4, 8, 16, 20])
        more["window"] = rng.choice([0, 0, 0, _spread(rng, 1, max(2, longest))])
    return {k: v for k, v in _cache("", op, b, hkv, d, page, longest, dtype, cache, order, **more).items() if k != "name"}


def _lens(case):
    """The sequences' lengths: the longest one first, the others spread down to a quarter of it; an empty and a one-token one in a batch."""
    rng = random.Random(1000003 * case["b"] + case["longest"])
    lens = [case["longest"]] + [rng.randint(max(1, case["longest"] // 4), case["longest"]) for _ in range(case["b"] - 1)]
    if case["b"] >= 5:
        lens[2] = 1
        if case["op"] != "append":
            lens[3] = 0
    return lens


def _fresh(case, lens):
    """New tokens of each sequence: one, or its last three quarters or so (a prompt behind a shared beginning)."""
    return [1] * len(lens) if case["new"] == 1 else [n - n // 4 for n in lens]


# ---------------------------------------------------------------------------- inputs
def _quantise(x):
    """e4m3 codes and scale bytes of float32 rows: the smallest power of two that brings the row's largest value to 448 or less."""
    fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    m, k = torch.frexp(fin)
    e = torch.where(fin == 0, torch.zeros_like(k), k - 9 + (m > 0.875)).clamp(-60, 127)
    y = torch.ldexp(x, -e[..., None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _frequencies(rot, far):
    """base^(-2i/rot), slowed down evenly where the positions go past 8192."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (10000.0 ** (-2.0 * i / rot) / max(1.0, far / 8192.0)).cuda()


def _values(gen, shape, dtype, d):
    """Rows as projections give them: unit values with a few channels several times as large."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype)
    lift = torch.ones(d, device="cuda", dtype=x.dtype)
    lift[torch.randperm(d, generator=gen, device="cuda")[: max(1, d // 32)]] = 4.0
    return x.mul_(lift)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    s = dict(case)
    dt = _TYPES[case["dtype"]]
    if case["op"] == "rope":
        b, h, n, d = case["b"], case["h"], case["n"], case["d"]
        if case["order"] == "bhnd":
            s["x"] = _values(gen, (b, h, n, d), dt, d)
        else:
            s["x"] = _values(gen, (b, n, h, d), dt, d).transpose(1, 2)
        s["y"] = torch.empty_like(s["x"])
        s["positions"] = torch.randint(0, max(1, case["far"] - n) + 1, (b, 1), generator=gen, device="cuda", dtype=torch.int32) + \
            torch.arange(n, device="cuda", dtype=torch.int32)
        s["inv_freq"], s["magnitude"] = _frequencies(case["rot"], case["far"]), 1.0 + 0.1 * math.log(max(1.0, case["far"] / 8192.0))
        return s
    lens = _lens(case)
    hkv, d, page = case["hkv"], case["d"], case["page"]
    wide = -(-max(lens) // page)
    pages = sum(-(-n // page) for n in lens) + 3
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).cpu()
    table, at = torch.zeros(case["b"], wide, dtype=torch.int32), 0
    for i, n in enumerate(lens):
        table[i, : -(-n // page)] = perm[at: at - (-n // page)]
        at += -(-n // page)
    s["table"], s["lens"] = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    shape = (pages, hkv, page, d) if case["order"] == "hnd" else (pages, page, hkv, d)
    for side in ("k", "v"):
        if case["cache"] == "e4m3":
            pool, exps = _quantise(_values(gen, shape, dt, d).float())
            s[side + "_exp"] = exps if case["order"] == "hnd" else exps.transpose(1, 2).contiguous()
        else:
            pool, s[side + "_exp"] = _values(gen, shape, dt, d), None
        s[side + "_pages"] = pool if case["order"] == "hnd" else pool.transpose(1, 2)
    if case["op"] == "append":
        new = _fresh(case, lens)
        total = sum(new)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu_new"] = None if case["new"] == 1 else torch.tensor(cu, dtype=torch.int32, device="cuda")
        # keys and values are slices of one projection's output
        kv = _values(gen, (total, 2 * hkv, d), dt, d)
        s["k"], s["v"] = kv[:, :hkv], kv[:, hkv:]
    elif case["op"] == "read":
        s["k_out"], s["v_out"] = (torch.zeros(case["b"], hkv, max(lens), d, device="cuda", dtype=dt) for _ in range(2))
    else:
        hq = hkv * case["group"]
        s["q"] = _values(gen, (case["b"], hq, d), dt, d)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["b"], hq, device="cuda", dtype=torch.float32)
        s["workspace"] = torch.empty(16 << 20, device="cuda", dtype=torch.uint8)
    return s


# ---------------------------------------------------------------------------- the plain forms
def _rotate(s):
    r = s["rot"] // 2
    angle = s["positions"].double()[:, None, :, None] * s["inv_freq"]
    cos = (angle.cos() * s["magnitude"]).float()
    sin = (angle.sin() * (s["magnitude"] if s["way"] == "forward" else -s["magnitude"])).float()
    x = s["x"].float()
    if s["pairs"] == "half":
        x1, x2 = x[..., :r], x[..., r:2 * r]
        y = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin, x[..., 2 * r:]], -1)
    else:
        x1, x2 = x[..., :2 * r:2], x[..., 1:2 * r:2]
        y = torch.cat([torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2), x[..., 2 * r:]], -1)
    return y.to(s["x"].dtype)


def _append(s):
    if s["cu_new"] is None:
        seq = torch.arange(s["b"], device="cuda")
        pos = s["lens"].long() - 1
    else:
        cu = s["cu_new"].long()
        t = torch.arange(s["k"].shape[0], device="cuda")
        seq = torch.searchsorted(cu[1:], t, right=True)
        pos = s["lens"].long()[seq] - cu[seq + 1] + t
    page, slot = s["table"].long()[seq, pos // s["page"]], pos % s["page"]
    kc, vc = s["k"], s["v"]
    if s["cache"] == "e4m3":
        kc, ke = _quantise(s["k"].float())
        vc, ve = _quantise(s["v"].float())
        s["k_exp"][page, :, slot], s["v_exp"][page, :, slot] = ke, ve
        s["k_pages"].view(torch.uint8)[page, :, slot], s["v_pages"].view(torch.uint8)[page, :, slot] = kc.view(torch.uint8), vc.view(torch.uint8)
    else:
        s["k_pages"][page, :, slot], s["v_pages"][page, :, slot] = kc, vc


def _gather(pool, exps, table):
    """[B, H, N, D] float32 rows of the sequences' pages."""
    t = table.long()
    x = pool.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() if exps is not None else pool[t].float()
    if exps is not None:
        x = torch.ldexp(x, exps[t].int()[..., None] - 127)
    b, j, h, p, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, j * p, d)


def _read(s):
    n = s["k_out"].shape[2]
    live = (torch.arange(n, device="cuda") < s["lens"][:, None])[:, None, :, None]
    k, v = (_gather(s[c + "_pages"], s[c + "_exp"], s["table"])[:, :, :n].to(s["k_out"].dtype) for c in ("k", "v"))
    s["k_out"].copy_(torch.where(live, k, s["k_out"]))
    s["v_out"].copy_(torch.where(live, v, s["v_out"]))


def _attend(s):
    k, v = (_gather(s[c + "_pages"], s[c + "_exp"], s["table"]) for c in ("k", "v"))
    n = k.shape[2]
    at, lens = torch.arange(n, device="cuda"), s["lens"][:, None]
    live = at < lens
    if s["window"]:
        live = live & (at >= lens - s["window"])
    live = live[:, None, None, :]
    q = s["q"].float().unflatten(1, (s["hkv"], s["group"]))
    score = (q @ k.transpose(-1, -2)) / math.sqrt(s["d"])
    score = score.masked_fill(~live, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ v.masked_fill(~live.transpose(-1, -2), 0.0)) / torch.where(total == 0, torch.ones_like(total), total)
    return o.flatten(1, 2).to(s["q"].dtype), (top + total.log())[..., 0].flatten(1, 2)


# ---------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    if s["op"] == "rope":
        return _rotate(s)
    if s["op"] == "append":
        _append(s)
        return _stored(s)
    if s["op"] == "read":
        _read(s)
        return s["k_out"], s["v_out"]
    return _attend(s)


def _stored(s):
    return {c: s[c] for c in ("k_pages", "v_pages", "k_exp", "v_exp") if s[c] is not None}


def _own(s):
    from attention_fa2_forward_02_gb300 import binding as fa2
    if s["op"] == "rope":
        call = fa2.fa2_rope if s["way"] == "forward" else fa2.fa2_rope_backward
        call(s["x"], s["y"], s["inv_freq"], positions=s["positions"], interleaved=s["pairs"] == "interleaved", magnitude=s["magnitude"])
        return s["y"]
    if s["op"] == "append":
        fa2.fa2_kv_append(s["k_pages"], s["v_pages"], s["k"], s["v"], s["table"], s["lens"], cu_new=s["cu_new"], k_exp=s["k_exp"],
                          v_exp=s["v_exp"])
        return _stored(s)
    if s["op"] == "read":
        fa2.fa2_kv_read(s["k_pages"], s["v_pages"], s["k_out"], s["v_out"], s["table"], s["lens"], k_exp=s["k_exp"], v_exp=s["v_exp"])
        return s["k_out"], s["v_out"]
    fa2.fa2_decode(s["q"], s["k_pages"], s["v_pages"], s["o"], s["lse"], s["table"], s["lens"], s["workspace"], 1 / math.sqrt(s["d"]),
                   window=s["window"], k_exp=s["k_exp"], v_exp=s["v_exp"])
    return s["o"], s["lse"]


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        n = case["b"] * case["h"] * case["n"]
        return {"bytes": 2 * n * case["d"] * size + case["b"] * case["n"] * 4 + case["rot"] * 4, "flops": 3 * n * case["rot"]}
    lens = _lens(case)
    row = case["hkv"] * case["d"]  # elements of a token's keys
    held = row + case["hkv"] if case["cache"] == "e4m3" else row * size
    if case["op"] == "append":
        n = sum(_fresh(case, lens))
        return {"bytes": 2 * n * (row * size + held), "flops": 2 * n * row * (2 if case["cache"] == "e4m3" else 0)}
    if case["op"] == "read":
        n = sum(lens)
        return {"bytes": 2 * n * (row * size + held), "flops": 2 * n * row * (1 if case["cache"] == "e4m3" else 0)}
    n = sum(min(x, case["window"]) if case["window"] else x for x in lens)
    q = case["b"] * row * case["group"]
    return {"bytes": 2 * n * held + 2 * q * size + q // case["d"] * 4, "flops": 4 * n * row * case["group"]}


# ---------------------------------------------------------------------------- the definitions in 64 bits
def _value64(codes, exps):
    """What e4m3 bytes stand for, from their bits: sign, 4 exponent bits (bias 7), 3 fraction bits; all ones is NaN."""
    c = codes.view(torch.uint8).to(torch.int64)
    e, f = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2((e - 7).double()))
    mag = torch.where((c & 127) == 127, torch.full_like(mag, math.nan), mag)
    return torch.where(c >= 128, -mag, mag) * torch.exp2(exps.double() - 127)[..., None]


def _code64(rows):
    """The e4m3 value nearest to each element of the rows at the row's scale (ties to the even fraction), and the scale bytes."""
    big = rows.abs().amax(-1)
    e = torch.where(big > 0, torch.ceil(torch.log2(big.clamp(min=1e-300) / 448.0)), torch.zeros_like(big))
    e = torch.where((big > 0) & (big <= 448.0 * torch.exp2(e - 1)), e - 1, e)
    e = torch.where(big > 448.0 * torch.exp2(e), e + 1, e).clamp(-60, 127)
    y = rows * torch.exp2(-e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, (e + 127).to(torch.uint8)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        r = case["rot"] // 2
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[:, None, :, None] * s["inv_freq"])
        turn = (turn if case["way"] == "forward" else turn.conj()) * s["magnitude"]
        x = s["x"].double()
        y = x.clone()
        one, two = (slice(0, r), slice(r, 2 * r)) if case["pairs"] == "half" else (slice(0, 2 * r, 2), slice(1, 2 * r, 2))
        z = torch.complex(x[..., one], x[..., two]) * turn
        y[..., one], y[..., two] = z.real, z.imag
        return y
    lens = _lens(case)
    if case["op"] == "append":
        out = {}
        for side in ("k", "v"):
            pool = s[side + "_pages"].double()
            rows = s[side].double()
            if case["cache"] == "e4m3":
                rows, exps = _code64(rows)
                out[side + "_exp"] = s[side + "_exp"].clone()
            at = 0
            for b, n in enumerate(_fresh(case, lens)):
                pos = torch.arange(lens[b] - n, lens[b], device="cuda")
                page, slot = s["table"][b].long()[pos // case["page"]], pos % case["page"]
                pool[page, :, slot] = rows[at: at + n]
                if case["cache"] == "e4m3":
                    out[side + "_exp"][page, :, slot] = exps[at: at + n]
                at += n
            out[side + "_pages"] = pool
        return out
    sides = []
    for side in ("k", "v"):
        rows = []
        for b, n in enumerate(lens):
            t = s["table"][b, : -(-n // case["page"])].long()
            pool = s[side + "_pages"]
            if case["cache"] == "e4m3":
                x = _value64(pool.view(torch.uint8)[t], s[side + "_exp"][t])
            else:
                x = pool[t].double()
            rows.append(x.transpose(1, 2).reshape(-1, case["hkv"], case["d"])[:n].transpose(0, 1))
        sides.append(rows)
    if case["op"] == "read":
        out = []
        for rows in sides:
            full = torch.zeros(case["b"], case["hkv"], max(lens), case["d"], dtype=torch.float64, device="cuda")
            for b, x in enumerate(rows):
                full[b, :, : lens[b]] = x
            out.append(full)
        return tuple(out)
    hq, d = case["hkv"] * case["group"], case["d"]
    o = torch.zeros(case["b"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["b"], hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n - first <= 0:
            continue
        k, v = sides[0][b][:, first:], sides[1][b][:, first:]
        q = s["q"][b].double().view(case["hkv"], case["group"], d)
        score = torch.einsum("hgd,hnd->hgn", q, k) / math.sqrt(d)
        lse[b] = torch.logsumexp(score, -1).flatten()
        o[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(score, -1), v).reshape(hq, d)
    return o, lse
