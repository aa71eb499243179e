"""Slots that hold no key may hold anything: pools that were never cleared, rows of sequences that are gone, in every byte of
theirs.  Tolerances are test_gpu_decode.py's."""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from tests import gpu_util as G
from tests.paged import Cache
from tests.paged4 import Cache4
from tests.test_gpu_decode import check, workspace
from tests.test_gpu_select import Selected, check_bounds, check_selection, make_bounds, select

pytestmark = pytest.mark.gpu


def unwritten(c):
    """Which rows [pages, n_kv_heads, page] no sequence has."""
    out = np.ones((c.pages, c.hkv, c.page), dtype=bool)
    for b, n in enumerate(c.lens):
        for pos in range(n):
            out[c.table[b, pos // c.page], :, pos % c.page] = False
    return out


def fill_unwritten(c, byte):
    """All bytes of those rows: `byte`, or (None) of any value, 255 and 0 among them."""
    import torch
    out = torch.from_numpy(unwritten(c)).cuda()
    for side in "kv":
        parts = [c.dev[side].view(torch.uint8), c.exp[side]] + ([c.scale[side].view(torch.uint8)] if hasattr(c, "scale") else [])
        for i, part in enumerate(parts):
            shape = tuple(part.shape)
            x = torch.full(shape, byte or 0, dtype=torch.uint8, device="cuda")
            if byte is None:
                x = torch.from_numpy((synth.counter_u16(f"unwritten/{side}/{i}", shape) >> 8).astype(np.uint8)).cuda()
            part[out] = x[out]
    return c


def cache(form, tag, lens, page, hkv, d, dtype="bf16", order="hnd", **kw):
    if form == "e2m1":
        return Cache4(tag, lens, page, hkv, d, dtype, order, stale=True, **kw)
    return Cache(tag, lens, page, hkv, d, dtype, True, order, **kw)


def decode(c, tag, group, window=0, rows=None):
    heads, scale = c.hkv * group, 1 / math.sqrt(c.d)
    q = synth.tensor(tag + "/q", (len(c.lens), heads, c.d), c.dtype)
    o, lse = G.guarded((len(c.lens), heads, c.d), c.dtype), G.guarded((len(c.lens), heads), "f32")
    binding.fa2_decode(G.to_device(q, c.dtype), *c.pools(), o.t, lse.t, c.table_dev, c.lens_dev, workspace(len(c.lens), heads, c.hkv, c.d), scale,
                       window=window, **c.exps())
    binding.fa2_device_status()
    o.assert_intact("O")
    lse.assert_intact("LSE")
    check(c, synth.widen(q, c.dtype), o.t, lse.t, group, scale, window, rows)


@pytest.mark.parametrize("byte", [255, 0, 254, None])
@pytest.mark.parametrize("d", [128, 96, 64, 32])
def test_head_sizes(d, byte):
    G.require_gpu()
    for dtype, order in (("bf16", "hnd"), ("f16", "nhd")):
        decode(fill_unwritten(cache("e2m1", f"unwritten/{d}", [37, 200, 1, 0], 16, 2, d, dtype, order), byte), f"unwritten/{d}", 4)


@pytest.mark.parametrize("form", ["e2m1", "e4m3"])
@pytest.mark.parametrize("page", [1, 8, 16, 24, 48, 64, 1024])
def test_page_sizes(page, form):
    G.require_gpu()
    for byte in (255, None):
        decode(fill_unwritten(cache(form, f"unwritten/p{page}", [150, 33, 64, 0, 7], page, 3, 64), byte), f"unwritten/p{page}", 2)


@pytest.mark.parametrize("group", [1, 8, 9, 16, 17])
def test_groups(group):
    G.require_gpu()
    decode(fill_unwritten(cache("e2m1", "unwritten/g", [70, 5], 16, 2, 128), 255), f"unwritten/g{group}", group)


@pytest.mark.parametrize("n", [1, 15, 17, 31, 33, 63, 65, 127, 129, 1000, 2049])
def test_lengths(n):
    G.require_gpu()
    for d in (128, 32):
        decode(fill_unwritten(cache("e2m1", f"unwritten/n{n}", [n], 16, 1, d), 255), f"unwritten/n{n}", 4)


@pytest.mark.parametrize("d", [128, 96, 64, 32])
def test_windows_and_rows_joined_from_many_ctas(d):
    """In one launch and in two; rows before the window count as little as those behind the length."""
    torch = G.require_gpu()
    for wide in (None, 2000):
        c = fill_unwritten(cache("e2m1", "unwritten/win", [200, 16, 17, 1, 0, 259], 16, 2, d, table_pages=wide), 255)
        for window in (0, 1, 17, 100):
            decode(c, "unwritten/win", 2, window)
        if window:  # the last one's
            before = torch.from_numpy(unwritten(c)).cuda()
            for b, n in enumerate(c.lens):
                for pos in range(max(0, n - window)):
                    before[c.table[b, pos // 16], :, pos % 16] = True
            for side in "kv":
                c.exp[side][before] = 255
                c.scale[side].view(torch.uint8)[before] = 0x7F
            decode(c, "unwritten/win", 2, window)
    decode(fill_unwritten(cache("e2m1", "unwritten/long", [5003], 16, 1, d), 255), "unwritten/long", 3)


@pytest.mark.parametrize("form", ["e2m1", "e4m3"])
@pytest.mark.parametrize("byte", [255, None])
def test_bounds_selection_and_its_attention(byte, form):
    torch = G.require_gpu()  # noqa: F841
    for d, page in ((128, 16), (64, 32), (96, 16), (32, 24)):
        hkv, group, budget = 2, 4, 5
        c = fill_unwritten(cache(form, f"unwritten/sel{d}", [300, 37, 1, 0, 161], page, hkv, d), byte)
        bounds, exps, cu = make_bounds(c)
        check_bounds(c, bounds, exps, cu)
        heads, scale = hkv * group, 1 / math.sqrt(d)
        full = synth.tensor("unwritten/sel/q", (5, heads, d), c.dtype)
        q, q64 = G.to_device(full, c.dtype), synth.widen(full, c.dtype)
        table, lens = select(c, q, bounds.t, exps.t, budget, 1, 1)
        taken = check_selection(c, q64, bounds.t.cpu().numpy().astype(np.int64), exps.t.cpu().numpy(), table, lens, budget, 1, 1)
        o, lse = G.empty((5, heads, d), c.dtype), torch.empty(5, heads, device="cuda")
        binding.fa2_decode_selected(q, *c.pools(), o, lse, table, lens, workspace(5, heads, hkv, d), scale, **c.exps())
        binding.fa2_device_status()
        for (b, h), want in taken.items():
            part = slice(h * group, (h + 1) * group)
            check(Selected(c, b, want).of_head(h), q64[b:b + 1, part], o[b:b + 1, part], lse[b:b + 1, part], group, scale)
