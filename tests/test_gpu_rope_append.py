"""Queries and keys turned, keys and values stored, in one call, against the float64 oracle.

Tolerance: a rotation's sine and cosine are within 3.4 2^-24, the product with the magnitude, the two products and their sum add
four roundings: a turned element is within r = 8 2^-24 |m| (|x1| + |x2|) of the oracle's y before its own rounding, which is
u |y| in 16 bits (2^-25 at most below half's smallest normals); in 8 bits 2^-4 |y|, or 2^-10 of the row's power of two; in 4 bits half a step of its scale s
(1/4, 1/2, 1 of it where |y| is below 2, 4, 6 of it, and what is above 6 s), with s within 2^-4 of a sixth of the 16 elements' largest, or
within 2^-10 of the row's power of two. The powers of two and everything about values are exact."""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.tolerance import UNIT_ROUNDOFF

pytestmark = pytest.mark.gpu

FORMS = ("same", "e4m3", "e2m1")


class Pages:
    """Pools of one form filled with a byte pattern."""

    def __init__(self, form, pages, hkv, page, d, dtype, order="hnd", fill=0x5A):
        import torch
        self.form, self.pages, self.hkv, self.page, self.d, self.dtype, self.fill = form, pages, hkv, page, d, dtype, fill
        row = {"same": 2 * d, "e4m3": d, "e2m1": d // 2}[form]
        shape = (pages, hkv, page, row) if order == "hnd" else (pages, page, hkv, row)
        raw = [torch.full(shape, fill, dtype=torch.uint8, device="cuda") for _ in "kv"]
        self.raw = [t if order == "hnd" else t.transpose(1, 2) for t in raw]
        view = {"same": getattr(torch, G.TORCH_DTYPE_NAMES[dtype]), "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}[form]
        self.pools = [t.view(view) if order == "hnd" else t.view(view).transpose(1, 2) for t in raw]
        byte = lambda *s: torch.full(s, fill, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.kw = {}
        if form != "same":
            self.kw |= {f"{s}_exp": byte(pages, hkv, page) for s in "kv"}
        if form == "e2m1":
            self.kw |= {f"{s}_scale": byte(pages, hkv, page, d // 16).view(torch.float8_e4m3fn) for s in "kv"}

    def row(self, side, at):
        """(values [d], byte, scales [d / 16]) of slot at = (page, head, slot)."""
        import torch
        raw = self.raw["kv".index(side)][at].cpu().numpy()
        if self.form == "same":
            return synth.widen(raw.view(np.uint16 if self.dtype == "bf16" else np.float16), self.dtype), None, None
        byte = int(self.kw[side + "_exp"][at].item())
        if self.form == "e4m3":
            return S.row_values(raw, byte), byte, None
        scales = self.kw[side + "_scale"].view(torch.uint8)[at].cpu().numpy()
        return S.row_values4(np.stack([raw & 15, raw >> 4], -1).reshape(-1), scales, byte), byte, S.e4m3_values()[scales] * 2.0 ** (byte - 127)

    def untouched(self, slots):
        """Whether everything but the given (page, slot) pairs is as it was."""
        import torch
        keep = torch.ones(self.pages, self.page, dtype=torch.bool, device="cuda")
        for _, pg, slot in slots:
            keep[pg, slot] = False
        m = keep[:, None].expand(self.pages, self.hkv, self.page)
        return all(bool((t[m] == self.fill).all()) for t in [*self.raw, *(x.view(torch.uint8) for x in self.kw.values())])


def check_row(form, dtype, got, byte, scales, y, before, r, more):
    """A stored key against its oracle y [d], of a row `before` its rotation; r: how far off the rotation itself may be."""
    if form == "same":
        assert np.all(np.abs(got - y) <= UNIT_ROUNDOFF[dtype] * (np.abs(y) + r) + r + 2.0 ** -25)
        return
    a = np.abs(before).max()
    if form == "e4m3":
        e = min((S.smallest_exp(a, 448.0) if a > 0 else 0) + more + 1, 120)
        assert byte == e + 127
        assert np.all(np.abs(got - y) <= r + np.maximum(2.0 ** -4 * (np.abs(y) + r), 2.0 ** (e - 10)))
        return
    e = S.quantise_row4(before)[2] - 127 + more
    assert byte == e + 127
    s = np.repeat(scales, 16)
    big = np.abs(y).reshape(-1, 16).max(1).repeat(16)
    top = r.reshape(-1, 16).max(1).repeat(16)
    assert np.all(np.abs(s - big / 6) <= 2.0 ** -4 * (big + top) / 6 + top + 2.0 ** (e - 10))
    step = np.where(np.abs(got) < 2 * s, 0.25, np.where(np.abs(got) < 4 * s, 0.5, 1.0)) * s
    over = np.maximum(np.abs(y) - 6 * s, 0)
    # a code on a border may lie in the wider step above
    step = np.maximum(step, np.where(np.abs(y) + r >= 4 * s, 1.0, np.where(np.abs(y) + r >= 2 * s, 0.5, 0.25)) * s)
    assert np.all(np.abs(got - y) <= r + np.maximum(step, over))


def run(tag, form, d, rot, dtype="bf16", interleaved=False, hkv=2, heads=3, page=16, order="hnd", new=(7, 0, 33, 1), before=(5, 3, 0, 40),
        magnitude=1.0, ones=False, positions=None, in_place=False, edit=None):
    torch = G.require_gpu()
    lens = [a + b for a, b in zip(new, before)]
    wide = -(-max(lens) // page)
    pages = len(lens) * wide + 2
    table = np.argsort(synth.raw_words(3, tag, 0, pages), kind="stable")[: len(lens) * wide].reshape(len(lens), wide).astype(np.int32)
    cu = None if ones else np.concatenate([[0], np.cumsum(new)]).astype(np.int32) + 2
    total = len(lens) if ones else int(cu[-1]) + 3
    p = Pages(form, pages, hkv, page, d, dtype, order)
    x = synth.tensor(f"{tag}/x", (total, heads + 2 * hkv + 1, d), dtype, scale=3.0)
    w = synth.widen(x, dtype)
    qkv = G.to_device(x, dtype)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + hkv], qkv[:, heads + hkv:heads + 2 * hkv]
    freq, _ = binding.fa2_rope_frequencies(rot, 10000.0)
    if edit:
        edit(table, lens)
    dev = lambda a: None if a is None else torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    out = G.guarded((total, heads, d), dtype)
    q_out = None if not heads else q if in_place else out.t
    pos_given = None if positions is None else dev(positions[:total])
    binding.fa2_rope_append(*p.pools, k, v, freq.cuda(), dev(table), dev(lens), q=q if heads else None, q_out=q_out, cu_new=dev(cu),
                            positions=pos_given, interleaved=interleaved, magnitude=magnitude, **p.kw)
    slots = S.append_slots(table, lens, cu, page, pages)
    # ---- which tokens have a position, and which
    place = {}
    for b, n in enumerate(lens):
        first, end = (b, b + 1) if cu is None else (cu[b], cu[b + 1])
        for t in range(first, end):
            pos = n - end + t
            if 0 <= pos < wide * page:
                place[t] = pos
    angle = np.array([[(positions[t] if positions is not None else place.get(t, 0)) for t in range(total)]])
    y = S.rope(w.transpose(1, 0, 2)[None], angle, freq.numpy(), interleaved, float(np.float32(magnitude)))[0].transpose(1, 0, 2)
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    r = np.zeros_like(w)
    r[..., one] = r[..., two] = 8 * 2.0 ** -24 * abs(magnitude) * (np.abs(w[..., one]) + np.abs(w[..., two]))
    more = max(0, math.ceil(math.log2(abs(magnitude)))) if magnitude else 0
    for t, pg, slot in slots:
        for h in range(hkv):
            got, byte, scales = p.row("k", (pg, h, slot))
            check_row(form, dtype, got, byte, scales, y[t, heads + h], w[t, heads + h], r[t, heads + h], more)
            got, byte, scales = p.row("v", (pg, h, slot))
            row = w[t, heads + hkv + h]
            ref = row if form == "same" else S.row_values(*S.quantise_row(row)) if form == "e4m3" else S.row_values4(*S.quantise_row4(row))
            assert np.array_equal(got, ref), (t, h)
    assert p.untouched(slots)
    if heads:
        got = G.to_f64(q_out)
        for t in range(total):
            if t in place:
                assert np.all(np.abs(got[t] - y[t, :heads]) <= UNIT_ROUNDOFF[dtype] * (np.abs(y[t, :heads]) + r[t, :heads]) + r[t, :heads] + 2.0 ** -25), t
            elif in_place:
                assert np.array_equal(got[t], w[t, :heads])
            else:
                assert np.isnan(got[t]).all()  # the pattern it was filled with
        out.assert_intact("q_out")
        if in_place:  # the other slices of the projection are only read
            assert torch.equal(qkv[:, heads:].view(torch.int16), G.to_device(x, dtype)[:, heads:].view(torch.int16))
    return p, slots


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 32), (64, 64), (64, 48), (32, 16), (96, 96), (96, 80), (96, 16), (128, 112)])
def test_heads_and_rotated_parts(d, rot, interleaved, form):
    run(f"ra/{d}/{rot}", form, d, rot, "bf16" if rot % 32 else "f16", interleaved)
    binding.fa2_device_status()


@pytest.mark.parametrize("d,rot,form", [(16, 16, "same"), (24, 16, "same"), (40, 32, "same"), (72, 64, "same"), (120, 112, "same"), (80, 80, "e4m3"),
                                        (16, 16, "e4m3"), (48, 48, "e4m3"), (112, 32, "e4m3")])
def test_odd_head_sizes(d, rot, form):
    run(f"ra/o{d}", form, d, rot, "f16", order="nhd")
    binding.fa2_device_status()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hkv,heads,page,order", [(1, 0, 16, "hnd"), (1, 1, 1, "nhd"), (8, 40, 24, "hnd"), (5, 15, 8, "nhd"), (16, 16, 64, "nhd"), (3, 33, 100, "hnd")])
def test_head_counts_and_pages(hkv, heads, page, order, form):
    run(f"ra/h{hkv}", form, 64, 32, hkv=hkv, heads=heads, page=page, order=order)
    binding.fa2_device_status()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("magnitude", [0.0, 0.3, 1.0, 1.35, 2.0, -5.0, 1000.0])
def test_magnitudes(magnitude, form):
    run("ra/mag", form, 64, 64, "bf16", magnitude=magnitude)
    binding.fa2_device_status()


@pytest.mark.parametrize("form", FORMS)
def test_one_token_a_sequence_far_positions_and_in_place(form):
    pos = [2 ** 31 - 1, -7, 1 << 20, 0, 65536, 12345]
    run("ra/step", form, 128, 128, new=(1,) * 6, before=(0, 15, 16, 700, 3, 99), ones=True, in_place=True)
    run("ra/step", form, 128, 64, new=(1,) * 6, before=(0, 15, 16, 700, 3, 99), ones=True, positions=pos)
    run("ra/pos", form, 64, 64, positions=list(range(100, 0, -1)), in_place=True)
    binding.fa2_device_status()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("tokens", [1300, 2500])
def test_many_tokens(tokens, form):
    """The ways a call divides its rows: whole tokens one by one, and four at a time."""
    run(f"ra/many{tokens}", form, 32, 32, hkv=1, heads=2, new=(tokens,), before=(3,))
    if tokens == 2500:
        run("ra/most", form, 32, 16, hkv=1, heads=1, new=(9000, 800), before=(0, 7), page=64)
    binding.fa2_device_status()


@pytest.mark.parametrize("form", FORMS)
def test_bad_pages_and_positions(form):
    def edit(table, lens):
        table[0, 0], table[2, 1] = 10 ** 6, -1  # turned, not stored
        lens[3] = 10 ** 6                       # no position: neither
    run("ra/bad", form, 64, 64, edit=edit)
    with pytest.raises(binding.Fa2Error) as err:
        binding.fa2_device_status()
    assert err.value.status == 8


@pytest.mark.parametrize("form", FORMS)
def test_nothing_for_an_empty_sequence(form):
    p, slots = run("ra/none", form, 64, 64, new=(1, 1, 1), before=(-1, 4, -1), ones=True)
    assert len(slots) == 1
    binding.fa2_device_status()


def test_infinities_and_nan_stay_in_their_pairs():
    """A NaN or an infinity reaches its own pair in 16 bits and in e4m3, its own 16 elements in 4 bits."""
    torch = G.require_gpu()
    for form in FORMS:
        p = Pages(form, 1, 1, 16, 64, "bf16")
        k = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
        k[0, 0, 3], k[1, 0, 40] = float("nan"), float("inf")
        freq, _ = binding.fa2_rope_frequencies(64, 10000.0)
        table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda")
        binding.fa2_rope_append(*p.pools, k, k, freq.cuda(), table, lens, cu_new=torch.tensor([0, 2], dtype=torch.int32, device="cuda"), **p.kw)
        binding.fa2_device_status()
        got = p.row("k", (0, 0, 0))[0]
        near = np.zeros(64, dtype=bool)
        near[[3, 35]] = True
        if form == "e2m1":
            near = near.reshape(-1, 16).any(1).repeat(16)
        assert np.isnan(got[near]).all() and np.isfinite(got[~near]).all() and np.all(np.abs(got[~near]) <= 1.6)
        got = p.row("k", (0, 0, 1))[0]
        # of a largest finite magnitude of 1: 448 of 2^(-8 + 1), 6 * 448 of 2^-9
        assert got[40] == {"same": np.inf, "e4m3": 448 * 2.0 ** -7, "e2m1": 2688 * 2.0 ** -9}[form] and np.isfinite(got[16:32]).all()
