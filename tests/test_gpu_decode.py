"""Attention of one new token over the paged cache, against the float64 oracle.

Tolerance, element by element, from the arithmetic. With u the rounding of the probabilities (2^-8 bfloat16, 2^-11 half;
half for e4m3), E = max_j scale sum_d |q_d k_jd| the largest score the terms allow:
 - a score's error is at most (d + 8) 2^-24 E: d products summed in float32, the scale, the scaling to base 2, the
   subtraction of the maximum; the exponential adds 2^-21;
 - each weight is rounded by u, and sums of n weights and products in float32 add n 2^-24;
 - both numerator and denominator carry the score errors: twice.
 - half's steps stop shrinking at 2^-24, so there a weight is off by up to 2^-25 instead. The weights are
   W_j = 2^(x_j - m), x_j = s_j log2(e) + e_j (e_j the value scale's exponent, 0 in a 16-bit cache), m no more than
   x_* = max x_j; O = sum W_j v_j 2^-e_j / sum W_j 2^-e_j, whose denominator is at least W_* 2^-e_* >= 2^-e_*: this
   moves O by at most 2^-25 sum_j |v_j| 2^(e_* - e_j).
So |O - ref| <= (u + 2 ((d + 8) 2^-24 E + 2^-21) + 2 n 2^-24) sum_j P_j |v_j| + [half] 2^-25 sum_j |v_j| 2^(e_* - e_j), and
half a step of the output. The LSE is within (d + 8) 2^-24 E + 2^-21 + n 2^-24 and its own rounding, 2^-23 (|ref| + E).
"""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.paged import Cache
from tests.tolerance import UNIT_ROUNDOFF

pytestmark = pytest.mark.gpu


def workspace(batch, heads, hkv, d, value=0xFF):
    import torch
    return torch.full((binding.fa2_decode_workspace_size(batch, heads, hkv, d),), value, dtype=torch.uint8, device="cuda")


def check(c, q64, o, lse, group, scale, window=0, rows=None):
    """Every (or the given) sequence and head of a decode call against the oracle; d-dimensional rows of c.dtype."""
    got_o, got_l = G.to_f64(o), G.to_f64(lse)
    u_out = UNIT_ROUNDOFF[c.dtype]
    u_p = UNIT_ROUNDOFF["f16" if c.e4m3 else c.dtype]
    for b in rows if rows is not None else range(len(c.lens)):
        k, held = c.rows("k", b)
        v, _ = c.rows("v", b)
        n = len(k)
        live = held & (np.arange(n) >= (n - window if window else 0))
        for h in range(q64.shape[1]):
            ref, rl, w, e = S.decode_row(q64[b, h], k[:, h // group], v[:, h // group], scale, live)
            if not live.any():
                assert not got_o[b, h].any() and got_l[b, h] == -np.inf
                continue
            score = (c.d + 8) * 2.0 ** -24 * e + 2.0 ** -21
            bound = (u_p + 2 * score + 2 * n * 2.0 ** -24) * w + u_out * np.abs(ref) + 2.0 ** -25
            if c.e4m3 or c.dtype == "f16":
                e_j = c.value_exps(b, h // group)[live]
                x = scale * (k[live, h // group] @ q64[b, h]) / math.log(2) + e_j
                bound = bound + 2.0 ** -25 * (2.0 ** (e_j[np.argmax(x)] - e_j) @ np.abs(v[live, h // group]))
            diff = np.abs(got_o[b, h] - ref)
            assert np.all(diff <= bound), f"sequence {b} (length {n}), head {h}: worst {np.max(diff - bound):.3e} past its bound"
            assert abs(got_l[b, h] - rl) <= score + n * 2.0 ** -24 + 2.0 ** -23 * (abs(rl) + e), f"LSE {b}, {h}: {got_l[b, h]} {rl}"


def run(tag, lens, page, hkv, group, d, dtype="bf16", e4m3=False, order="hnd", window=0, stale=None, q_scale=1.0, rows=None, **kw):
    torch = G.require_gpu()
    c = Cache(tag, lens, page, hkv, d, dtype, e4m3, order, stale=stale, **kw)
    heads = hkv * group
    # q as a slice of a wider projection
    full = synth.tensor(tag + "/q", (len(lens), heads + 2, d), dtype, scale=q_scale)
    q = G.to_device(full, dtype)[:, 1:heads + 1]
    o, lse = G.guarded((len(lens), heads, d), dtype), G.guarded((len(lens), heads), "f32")
    scale = 1 / math.sqrt(d)
    binding.fa2_decode(q, *c.pools(), o.t, lse.t, c.table_dev, c.lens_dev, workspace(len(lens), heads, hkv, d), scale, window=window,
                       **c.exps())
    binding.fa2_device_status()
    o.assert_intact("O")
    lse.assert_intact("LSE")
    check(c, synth.widen(full, dtype)[:, 1:heads + 1], o.t, lse.t, group, scale, window, rows)
    return c, q, o.t, lse.t


@pytest.mark.parametrize("dtype,e4m3", [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)])
@pytest.mark.parametrize("d", [128, 64, 32, 16, 80, 112])
def test_head_sizes_and_types(d, dtype, e4m3):
    run(f"decode/{d}", [37, 200, 1], 16, 2, 4, d, dtype, e4m3, stale="nan")


@pytest.mark.parametrize("d", [8, 24, 40, 72, 104, 120])
def test_head_sizes_of_half_chunks(d):
    run(f"decode/{d}", [37, 200, 1], 16, 2, 4, d, "f16", stale="inf")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 9, 16, 17, 20, 33])
def test_groups(group, e4m3):
    run(f"decode/g{group}", [70, 5], 16, 2, group, 64, "bf16", e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("order", ["hnd", "nhd"])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 100, 1000])
def test_page_sizes(page, order, e4m3):
    run(f"decode/p{page}", [150, 33, 64, 0, 7], page, 3, 2, 32, "f16", e4m3, order, stale="nan")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [0, 1, 2, 7, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 257, 1000, 2047, 2049])
def test_lengths(n, e4m3):
    run(f"decode/n{n}", [n], 16, 1, 4, 128, "bf16", e4m3, stale="nan")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("wide", [None, 2000])
@pytest.mark.parametrize("batch,hkv,group", [(1, 1, 1), (1, 8, 4), (3, 2, 16), (9, 8, 3), (70, 8, 2)])
def test_short_rows_in_one_launch_and_in_two(batch, hkv, group, wide, e4m3):
    """A narrow block table takes the clusters of one launch (of 8, 4, 2 CTAs and of one, as the items grow), a wide one
    with the same lengths the two launches; empty sequences, shares without a block and windows among them."""
    lens = [(37 * i * i + 5 * i) % 260 for i in range(batch)]
    lens[0] = 259
    run("decode/short", lens, 16, hkv, group, 64, "bf16", e4m3, stale="nan", table_pages=wide, rows=range(0, batch, 7))
    run("decode/short", lens, 16, hkv, group, 128, "f16", e4m3, "nhd", window=77, table_pages=wide, rows=range(0, batch, 7))


@pytest.mark.parametrize("e4m3", [False, True])
def test_long_rows_joined_from_many_ctas(e4m3):
    run("decode/long", [20000], 16, 1, 3, 64, "bf16", e4m3)
    run("decode/long2", [9000, 1, 5000], 64, 2, 8, 128, "f16", e4m3, "nhd")


@pytest.mark.parametrize("e4m3", [False, True])
def test_large_batches_of_ragged_lengths(e4m3):
    """More sequences than a CTA has threads, empty ones among them and at both ends."""
    lens = [0, 0] + [int(x % 50) for x in synth.raw_words(5, "decode/ragged", 0, 700)] + [0]
    run("decode/ragged", lens, 8, 1, 2, 32, "bf16", e4m3, stale="nan")


def test_all_empty():
    run("decode/empty", [0, 0, 0], 16, 2, 2, 64)


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 199, 200, 1 << 40])
@pytest.mark.parametrize("e4m3", [False, True])
def test_window(window, e4m3):
    run("decode/win", [200, 16, 17, 1, 0], 16, 2, 2, 64, "bf16", e4m3, "nhd", window=window, stale="nan")


@pytest.mark.parametrize("e4m3", [False, True])
def test_peaked_scores(e4m3):
    """Scores of some hundreds: one key takes all, the running maximum moves often."""
    run("decode/peak", [500, 33], 16, 2, 4, 64, "f16", e4m3, q_scale=40.0)


def test_values_of_very_different_scales():
    """e4m3 rows whose scales differ by 2^40: the small rows do not count, the large ones are exact."""
    torch = G.require_gpu()
    c = Cache("decode/scales", [64], 16, 1, 32, "bf16", True)
    for s, low, high in (("k", 100, 120), ("v", 90, 130)):
        e = np.where(np.arange(c.pages * 16).reshape(c.pages, 1, 16) % 5 == 0, high, low).astype(np.uint8)
        codes = c.dev[s].contiguous().view(torch.uint8).cpu().numpy()
        c.exp[s].copy_(torch.from_numpy(e))
        c.host[s] = S.e4m3_values()[codes] * 2.0 ** (e[..., None].astype(np.float64) - 127)
    q = synth.tensor("decode/scales/q", (1, 2, 32), "bf16")
    o, lse = G.empty((1, 2, 32), "bf16"), torch.empty(1, 2, device="cuda")
    binding.fa2_decode(G.to_device(q, "bf16"), *c.pools(), o, lse, c.table_dev, c.lens_dev, workspace(1, 2, 1, 32), 0.2, **c.exps())
    check(c, synth.widen(q, "bf16"), o, lse, 2, 0.2)


def test_minus_infinity_and_nan_in_live_rows():
    """A NaN in a live key spreads to its heads, not to other sequences."""
    torch = G.require_gpu()
    c = Cache("decode/nan", [40, 40], 16, 1, 32)
    c.dev["k"][c.table[1, 1], 0, 3, 5] = float("nan")
    q = synth.tensor("decode/nan/q", (2, 2, 32), "bf16")
    o, lse = G.empty((2, 2, 32), "bf16"), torch.empty(2, 2, device="cuda")
    binding.fa2_decode(G.to_device(q, "bf16"), *c.pools(), o, lse, c.table_dev, c.lens_dev, workspace(2, 2, 1, 32), 0.2)
    check(c, synth.widen(q, "bf16"), o, lse, 2, 0.2, rows=[0])
    assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_bad_pages_are_masked(e4m3):
    torch = G.require_gpu()
    lens = [100, 40, 16]
    c = Cache("decode/bad", lens, 16, 2, 64, "bf16", e4m3)
    c.table[0, 2], c.table[1, 0], c.table[2, 0] = c.pages, -1, 2 ** 31 - 1  # the last one leaves its row empty
    c.table_dev.copy_(torch.from_numpy(c.table))
    q = synth.tensor("decode/bad/q", (3, 4, 64), "bf16")
    o, lse = G.empty((3, 4, 64), "bf16"), torch.empty(3, 4, device="cuda")
    call = lambda: binding.fa2_decode(G.to_device(q, "bf16"), *c.pools(), o, lse, c.table_dev, c.lens_dev,  # noqa: E731
                                      workspace(3, 4, 2, 64), 0.125, **c.exps())
    call()
    with pytest.raises(binding.Fa2Error) as err:
        binding.fa2_device_status()
    assert err.value.status == 8
    check(c, synth.widen(q, "bf16"), o, lse, 2, 0.125)
    # lengths outside the table count as nothing, or as the whole table
    c.table[:] = np.arange(c.table.size).reshape(c.table.shape) % c.pages
    c.table_dev.copy_(torch.from_numpy(c.table))
    c.lens = [-5, 1000, 2 ** 31 - 1]
    c.lens_dev.copy_(torch.tensor(c.lens, dtype=torch.int32))
    call()
    with pytest.raises(binding.Fa2Error):
        binding.fa2_device_status()
    check(c, synth.widen(q, "bf16"), o, lse, 2, 0.125)


@pytest.mark.parametrize("e4m3", [False, True])
def test_offsets_past_2_32_bytes(e4m3):
    torch = G.require_gpu()
    c = Cache("decode/far", [60, 33], 16, 2, 64, "bf16", e4m3)
    size = 1 if e4m3 else 2
    stride = ((1 << 32) + 4096) // size // (c.pages - 1) // 64 * 64 + 64
    pools = []
    for s in "kv":
        small = c.dev[s].contiguous().view(torch.uint8) if e4m3 else c.dev[s].contiguous()
        buf = torch.zeros((c.pages - 1) * stride + 2 * 16 * 64, dtype=small.dtype, device="cuda")
        far = buf.as_strided((c.pages, 2, 16, 64), (stride, 16 * 64, 64, 1))
        far.copy_(small)
        pools.append(far.view(torch.float8_e4m3fn) if e4m3 else far)
    q = synth.tensor("decode/far/q", (2, 4, 64), "bf16")
    o, lse = G.empty((2, 4, 64), "bf16"), torch.empty(2, 4, device="cuda")
    binding.fa2_decode(G.to_device(q, "bf16"), *pools, o, lse, c.table_dev, c.lens_dev, workspace(2, 4, 2, 64), 0.125, **c.exps())
    binding.fa2_device_status()
    check(c, synth.widen(q, "bf16"), o, lse, 2, 0.125)


def test_same_bits_again():
    """Same inputs, workspace contents and run: the same bits; another workspace content changes nothing."""
    torch = G.require_gpu()
    c, q, o, lse = run("decode/again", [3000, 77, 900], 16, 2, 4, 128)
    for fill in (0, 0x7F):
        o2, l2 = torch.empty_like(o), torch.empty_like(lse)
        binding.fa2_decode(q, *c.pools(), o2, l2, c.table_dev, c.lens_dev, workspace(3, 8, 2, 128, fill), 1 / math.sqrt(128))
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_two_streams_at_once():
    torch = G.require_gpu()
    c, q, o, lse = run("decode/streams", [5000, 77, 900], 16, 2, 4, 64)
    outs = []
    main = torch.cuda.current_stream()
    for _ in range(4):
        side = torch.cuda.Stream()
        ws = workspace(3, 8, 2, 64)
        o2, l2 = torch.full_like(o, float("nan")), torch.full_like(lse, float("nan"))
        side.wait_stream(main)
        binding.fa2_decode(q, *c.pools(), o2, l2, c.table_dev, c.lens_dev, ws, 1 / math.sqrt(64), stream=side)
        outs.append((side, ws, o2, l2))
    torch.cuda.synchronize()
    for _, _, o2, l2 in outs:
        assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("group,d", [(1, 32), (8, 128), (16, 64), (12, 128)])
def test_workspace_of_exactly_the_size_asked_for(group, d, e4m3):
    """Rows divided between all the CTAs write every partial result; nothing lands outside the workspace."""
    torch = G.require_gpu()
    c = Cache("decode/ws", [9000, 4000], 64, 2, d, "bf16", e4m3)
    q = synth.tensor("decode/ws/q", (2, 2 * group, d), "bf16")
    o, lse = G.empty((2, 2 * group, d), "bf16"), torch.empty(2, 2 * group, device="cuda")
    ws = G.Guarded((binding.fa2_decode_workspace_size(2, 2 * group, 2, d),), torch.uint8)
    for n in ((9000, 4000), (0, 9000), (9000, 0), (300, 9000)):
        c.lens = list(n)
        c.lens_dev.copy_(torch.tensor(n, dtype=torch.int32))
        c.table[:] = np.arange(c.table.size).reshape(c.table.shape) % c.pages
        c.table_dev.copy_(torch.from_numpy(c.table))
        binding.fa2_decode(G.to_device(q, "bf16"), *c.pools(), o, lse, c.table_dev, c.lens_dev, ws.t, 1 / math.sqrt(d), **c.exps())
        binding.fa2_device_status()
        ws.assert_intact("workspace")
    check(c, synth.widen(q, "bf16"), o, lse, group, 1 / math.sqrt(d), rows=[0])


def test_many_sequences():
    """Far more sequences than threads and CTAs, most of them empty, and the largest batch a call takes."""
    torch = G.require_gpu()
    for batch in (5000, 65535):
        lens = np.zeros(batch, dtype=np.int64)
        at = [0, 1, 127, 128, batch // 2, batch - 2, batch - 1]
        lens[at] = [3, 40, 17, 5, 100, 16, 33]
        c = Cache("decode/many", [int(lens[i]) for i in at], 16, 1, 32, "bf16", True)
        table = torch.zeros(batch, c.wide, dtype=torch.int32, device="cuda")
        table[at] = c.table_dev
        q = synth.tensor("decode/many/q", (len(at), 2, 32), "bf16")
        full = torch.zeros(batch, 2, 32, dtype=torch.bfloat16, device="cuda")
        full[at] = G.to_device(q, "bf16")
        o, lse = torch.full_like(full, float("nan")), torch.full((batch, 2), float("nan"), device="cuda")
        binding.fa2_decode(full, *c.pools(), o, lse, table, torch.from_numpy(lens).int().cuda(), workspace(batch, 2, 1, 32), 0.2, **c.exps())
        binding.fa2_device_status()
        check(c, synth.widen(q, "bf16"), o[at], lse[at], 2, 0.2)
        rest = torch.ones(batch, dtype=torch.bool)
        rest[at] = False
        assert not o[rest].any() and bool((lse[rest] == -math.inf).all())
