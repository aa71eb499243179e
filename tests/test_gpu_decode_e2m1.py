"""Attention of one new token over a cache of 4-bit rows, against the float64 oracle.

The tolerance is test_gpu_decode.py's for an 8-bit cache, and holds for the same reasons: a row's values are its codes times its
scales, exact in half (6 bits), so that the arithmetic from there on, and the powers of two of the rows, are the same."""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.paged4 import Cache4
from tests.test_gpu_decode import check, workspace

pytestmark = pytest.mark.gpu


def run(tag, lens, page, hkv, group, d, dtype="bf16", order="hnd", window=0, stale=True, q_scale=1.0, rows=None, **kw):
    torch = G.require_gpu()  # noqa: F841
    c = Cache4(tag, lens, page, hkv, d, dtype, order, stale=stale, **kw)
    heads = hkv * group
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


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("order", ["hnd", "nhd"])
@pytest.mark.parametrize("d", [128, 96, 64, 32])
def test_head_sizes_and_types(d, order, dtype):
    run(f"decode4/{d}", [37, 200, 1], 16, 2, 4, d, dtype, order)


@pytest.mark.parametrize("d", [128, 96, 64, 32])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 48, 100, 1000])
def test_page_sizes(page, d):
    run(f"decode4/p{page}", [150, 33, 64, 0, 7], page, 3, 2, d, "f16", "nhd" if page % 2 else "hnd")


@pytest.mark.parametrize("d", [128, 32])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 9, 16, 17, 20, 33])
def test_groups(group, d):
    run(f"decode4/g{group}", [70, 5], 16, 2, group, d)


@pytest.mark.parametrize("n", [0, 1, 2, 7, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 2047, 2049])
def test_lengths(n):
    run(f"decode4/n{n}", [n], 16, 1, 4, 128)


@pytest.mark.parametrize("wide", [None, 2000])
@pytest.mark.parametrize("batch,hkv,group", [(1, 1, 1), (1, 8, 4), (3, 2, 16), (9, 8, 3), (70, 8, 2)])
def test_short_rows_in_one_launch_and_in_two(batch, hkv, group, wide):
    lens = [(37 * i * i + 5 * i) % 260 for i in range(batch)]
    lens[0] = 259
    run("decode4/short", lens, 16, hkv, group, 64, "bf16", table_pages=wide, rows=range(0, batch, 7))
    run("decode4/short", lens, 16, hkv, group, 128, "f16", "nhd", window=77, table_pages=wide, rows=range(0, batch, 7))


def test_long_rows_joined_from_many_ctas():
    run("decode4/long", [20000], 16, 1, 3, 64)
    run("decode4/long2", [9000, 1, 5000], 64, 2, 8, 128, "f16", "nhd")
    run("decode4/long3", [7000, 3], 24, 1, 8, 32)


@pytest.mark.parametrize("d,page", [(128, 16), (96, 16), (96, 24), (64, 16), (32, 16), (32, 8)])
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 199, 200, 1 << 40])
def test_window(window, d, page):
    run("decode4/win", [200, 16, 17, 1, 0], page, 2, 2, d, "bf16", "nhd", window=window)


def test_peaked_scores():
    run("decode4/peak", [500, 33], 16, 2, 4, 64, "f16", q_scale=40.0)


def test_rows_of_zeros_and_scales_far_apart():
    """Keys of very small values beside rows of zeros, whose power of two is far above the others'."""
    torch = G.require_gpu()
    c = Cache4("decode4/zeros", [300], 16, 1, 64)
    for side, low, high in (("k", 100, 120), ("v", 70, 100)):
        e = np.where(np.arange(c.pages * 16).reshape(c.pages, 1, 16) % 5 == 0, high, low).astype(np.uint8)
        zero = np.arange(c.pages * 16).reshape(c.pages, 1, 16) % 3 == 0
        if side == "v":
            c.codes[side][zero] = 0
            e[zero] = 127
        scales = c.scale[side].view(torch.uint8).cpu().numpy()
        c.host[side] = S.row_values4(c.codes[side], scales, e)
        c.dev[side].copy_(torch.from_numpy(S.pack4(c.codes[side])))
        c.exp[side].copy_(torch.from_numpy(e))
    q = synth.tensor("decode4/zeros/q", (1, 2, 64), "bf16")
    o, lse = G.empty((1, 2, 64), "bf16"), torch.empty(1, 2, device="cuda")
    binding.fa2_decode(G.to_device(q, "bf16"), *c.pools(), o, lse, c.table_dev, c.lens_dev, workspace(1, 2, 1, 64), 0.2, **c.exps())
    n = 300
    k, v = c.rows("k", 0)[0][:, 0], c.rows("v", 0)[0][:, 0]
    for h in range(2):
        ref, rl, w, e = S.decode_row(synth.widen(q, "bf16")[0, h], k, v, 0.2)
        # weights within 2^-11 each, sums of n in float32; and a half's smallest step beside the largest weight, which is a
        # row's that is not all zeros: each |v_j| counts with no more than 2^-25 of it
        score = (64 + 8) * 2.0 ** -24 * e + 2.0 ** -21
        live = np.abs(v).sum(1) > 0
        x = 0.2 * (k @ synth.widen(q, "bf16")[0, h]) / math.log(2) + c.value_exps(0, 0)
        e_j = c.value_exps(0, 0)
        top = e_j[live][np.argmax(x[live])]
        bound = (2.0 ** -11 + 2 * score + 2 * n * 2.0 ** -24) * w + 2.0 ** -8 * np.abs(ref) + 2.0 ** -25 * (2.0 ** (top - e_j[live]) @ np.abs(v[live]))
        assert np.all(np.abs(G.to_f64(o)[0, h] - ref) <= bound + 1e-38)
        assert abs(float(lse[0, h]) - rl) <= score + n * 2.0 ** -24 + 2.0 ** -23 * (abs(rl) + e)


def test_nan_scale_in_a_live_row_spreads_no_further():
    torch = G.require_gpu()
    c = Cache4("decode4/nan", [40, 40], 16, 1, 32)
    c.scale["k"].view(torch.uint8)[c.table[1, 1], 0, 3, 1] = 0x7F
    q = synth.tensor("decode4/nan/q", (2, 2, 32), "bf16")
    o, lse = G.empty((2, 2, 32), "bf16"), torch.empty(2, 2, device="cuda")
    binding.fa2_decode(G.to_device(q, "bf16"), *c.pools(), o, lse, c.table_dev, c.lens_dev, workspace(2, 2, 1, 32), 0.2, **c.exps())
    check(c, synth.widen(q, "bf16"), o, lse, 2, 0.2, rows=[0])
    assert torch.isnan(lse[1]).all()


def test_bad_pages_are_masked():
    torch = G.require_gpu()
    for d in (128, 96):
        c = Cache4("decode4/bad", [100, 40, 16], 16, 2, d)
        c.table[0, 2], c.table[1, 0], c.table[2, 0] = c.pages, -1, 2 ** 31 - 1
        c.table_dev.copy_(torch.from_numpy(c.table))
        q = synth.tensor("decode4/bad/q", (3, 4, d), "bf16")
        o, lse = G.empty((3, 4, d), "bf16"), torch.empty(3, 4, device="cuda")
        binding.fa2_decode(G.to_device(q, "bf16"), *c.pools(), o, lse, c.table_dev, c.lens_dev, workspace(3, 4, 2, d), 0.125, **c.exps())
        with pytest.raises(binding.Fa2Error) as err:
            binding.fa2_device_status()
        assert err.value.status == 8
        check(c, synth.widen(q, "bf16"), o, lse, 2, 0.125)


def test_offsets_past_2_32_bytes():
    torch = G.require_gpu()
    c = Cache4("decode4/far", [60, 33], 16, 2, 64)
    stride = ((1 << 32) + 4096) // (c.pages - 1) // 64 * 64 + 64
    pools = []
    for s in "kv":
        buf = torch.zeros((c.pages - 1) * stride + 2 * 16 * 32, dtype=torch.uint8, device="cuda")
        far = buf.as_strided((c.pages, 2, 16, 32), (stride, 16 * 32, 32, 1))
        far.copy_(c.dev[s])
        pools.append(far)
    q = synth.tensor("decode4/far/q", (2, 4, 64), "bf16")
    o, lse = G.empty((2, 4, 64), "bf16"), torch.empty(2, 4, device="cuda")
    binding.fa2_decode(G.to_device(q, "bf16"), *pools, o, lse, c.table_dev, c.lens_dev, workspace(2, 4, 2, 64), 0.125, **c.exps())
    binding.fa2_device_status()
    check(c, synth.widen(q, "bf16"), o, lse, 2, 0.125)


def test_offsets_past_2_36_bytes():
    """Pages further apart than 32 bits of 16 bytes reach."""
    torch = G.require_gpu()
    free, _ = torch.cuda.mem_get_info()
    stride = (1 << 35) + (1 << 30)
    if free < 2 * stride + (16 << 30):
        pytest.skip("not enough memory for two far pages")
    c = Cache4("decode4/farther", [30, 16], 16, 2, 64, spare=0)
    buf = torch.empty(2 * stride + 2 * 2 * 16 * 32, dtype=torch.uint8, device="cuda")
    pools = []
    for i, s in enumerate("kv"):  # K's and V's pages side by side in one buffer
        far = buf[i * 2 * 16 * 32:].as_strided((c.pages, 2, 16, 32), (stride, 16 * 32, 32, 1))
        far.copy_(c.dev[s])
        pools.append(far)
    q = synth.tensor("decode4/farther/q", (2, 4, 64), "bf16")
    o, lse = G.empty((2, 4, 64), "bf16"), torch.empty(2, 4, device="cuda")
    binding.fa2_decode(G.to_device(q, "bf16"), *pools, o, lse, c.table_dev, c.lens_dev, workspace(2, 4, 2, 64), 0.125, **c.exps())
    binding.fa2_device_status()
    check(c, synth.widen(q, "bf16"), o, lse, 2, 0.125)


def test_same_bits_again_and_on_another_stream():
    torch = G.require_gpu()
    c, q, o, lse = run("decode4/again", [3000, 77, 900], 16, 2, 4, 128)
    for fill in (0, 0x7F):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        o2, l2, ws = torch.full_like(o, 7.0), torch.empty_like(lse), workspace(3, 8, 2, 128, fill)
        torch.cuda.synchronize()
        binding.fa2_decode(q, *c.pools(), o2, l2, c.table_dev, c.lens_dev, ws, 1 / math.sqrt(128), stream=side, **c.exps())
        side.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("group,d", [(1, 32), (8, 128), (16, 64), (12, 128)])
def test_workspace_of_exactly_the_size_asked_for(group, d):
    torch = G.require_gpu()
    c = Cache4("decode4/ws", [9000, 4000], 64, 2, d)
    q = synth.tensor("decode4/ws/q", (2, 2 * group, d), "bf16")
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
