"""Value rows of an 8-bit cache whose scales lie far apart, in the attention of one new token: against the float64 oracle."""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.paged import Cache
from tests.test_gpu_decode import check, workspace
from tests.tolerance import UNIT_ROUNDOFF

pytestmark = pytest.mark.gpu

ONE, FOURTEEN = 0x38, 0x56  # e4m3 codes


def fill(c, side, codes=None, exps=None):
    """Sets the codes [tokens, d] and scale exponents [tokens] of sequence 0's rows, for every head."""
    import torch
    dev = c.dev[side].contiguous().view(torch.uint8).cpu().numpy()
    byte = c.exp[side].cpu().numpy()
    for pos in range(c.lens[0]):
        at = (c.table[0, pos // c.page], slice(None), pos % c.page)
        if codes is not None:
            dev[at] = codes[pos]
        if exps is not None:
            byte[at] = exps[pos] + 127
    c.dev[side] = torch.from_numpy(dev).cuda().view(torch.float8_e4m3fn)
    c.exp[side].copy_(torch.from_numpy(byte))
    c.host[side] = S.e4m3_values()[dev] * 2.0 ** (byte[..., None].astype(np.float64) - 127)


def attend(c, q, scale, heads):
    import torch
    o, lse = G.empty((1, heads, c.d), c.dtype), torch.empty(1, heads, device="cuda")
    binding.fa2_decode(G.to_device(q, c.dtype), *c.pools(), o, lse, c.table_dev, c.lens_dev, workspace(1, heads, c.hkv, c.d), scale, **c.exps())
    binding.fa2_device_status()
    return o, lse


# length, place of the one large value row: in one lane's keys, another lane's, another warp's, another CTA's
PLACES = [(2, 1), (33, 20), (64, 3), (400, 333), (20000, 0), (20000, 17003)]


@pytest.mark.parametrize("d,group", [(32, 2), (64, 12), (128, 4)])
@pytest.mark.parametrize("wide", [None, 2000])
@pytest.mark.parametrize("n,at", PLACES)
def test_rows_of_small_values_count_in_the_denominator(n, at, wide, d, group):
    """Value scales 2^-60 and 2^70: all keys have the same score, so O is the large row / n and the LSE ln n; and 2^-40 beside a
    2^110 that is e^14 times less likely.  (One key of the other scale, wherever it lies.)"""
    G.require_gpu()
    c = Cache("e4m3/apart", [n], 16, 1, d, "bf16", True, table_pages=max(wide or 0, -(-n // 16)) if wide else None)
    e = np.full(n, -60)
    e[at] = 70
    fill(c, "v", exps=e)
    zero = synth.to_storage(np.zeros((1, group, d)), "bf16")
    o, lse = attend(c, zero, 1 / math.sqrt(d), group)
    check(c, np.zeros((1, group, d)), o, lse, group, 1 / math.sqrt(d))

    e = np.full(n, -40)
    e[at] = 110
    likely = np.full((n, d), FOURTEEN, dtype=np.uint8)
    likely[at] = 0
    fill(c, "v", exps=e)
    fill(c, "k", likely, np.zeros(n, dtype=int))
    ones = synth.to_storage(np.ones((1, group, d)), "bf16")
    o, lse = attend(c, ones, 1 / d, group)
    check(c, np.ones((1, group, d)), o, lse, group, 1 / d)


def appended(tag, k, v, page=16, table_pages=None):
    """A cache of one sequence, its rows k, v [tokens, 1, d] (bf16 storage) written by fa2_kv_append."""
    import torch
    n, _, d = k.shape
    c = Cache(tag, [n], page, 1, d, "bf16", True, table_pages=table_pages)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    binding.fa2_kv_append(*c.pools(), G.to_device(k, "bf16"), G.to_device(v, "bf16"), c.table_dev, c.lens_dev, cu_new=cu, **c.exps())
    for side in "kv":
        codes = c.dev[side].contiguous().view(torch.uint8).cpu().numpy()
        c.host[side] = S.e4m3_values()[codes] * 2.0 ** (c.exp[side].cpu().numpy()[..., None].astype(np.float64) - 127)
    return c


def check_closely(c, q64, o, lse, scale, group=1):
    """As test_gpu_decode.check for sequence 0, but with the weights' rounding in two parts, and the weights that set the maximum
    those of rows with an element that is not 0.  A weight W_j = 2^(s_j + e_j) goes into the product as two 16-bit numbers, the
    second the rounded rest of the first: off by u^2 W_j, u the type's roundoff (from an 8-bit cache to bfloat16 results only
    the first: u W_j, u half's).  In half also by half a step of 2^-24 of a
    reference that is 2^7 below the largest weight W_* or lower: 2^-32 W_*, so O, whose denominator is L = sum 2^s_j, by
    (2^-32 W_* / L) sum_j |v_j| 2^-e_j."""
    half = c.e4m3 or c.dtype == "f16"
    u = UNIT_ROUNDOFF["f16" if half else "bf16"]
    step = u if c.e4m3 and c.dtype == "bf16" else u ** 2
    for h in range(q64.shape[1]):
        k, v = c.rows("k", 0)[0][:, h // group], c.rows("v", 0)[0][:, h // group]
        e_j, n = c.value_exps(0, h // group), len(k)
        ref, rl, w, e = S.decode_row(q64[0, h], k, v, scale)
        s = scale * (k @ q64[0, h]) / math.log(2)
        top = s.max()
        filled = np.abs(v).max(1) > 0
        largest = np.exp2((s + e_j)[filled].max() - top) if half and filled.any() else 0.0
        floor = 2.0 ** -32 * largest / np.exp2(s - top).sum() * (np.exp2(-e_j) @ np.abs(v))
        score = (c.d + 8) * 2.0 ** -24 * e + 2.0 ** -21
        bound = (step + 2 * score + 2 * n * 2.0 ** -24) * w + floor + UNIT_ROUNDOFF[c.dtype] * np.abs(ref)
        if c.dtype == "f16":
            bound = bound + 2.0 ** -25  # half a step of the smallest halves
        diff = np.abs(G.to_f64(o)[0, h] - ref)
        assert np.all(diff <= bound), f"head {h}: worst {np.max(diff / np.maximum(bound, 1e-300)):.3g} times its bound"
        assert abs(G.to_f64(lse)[0, h] - rl) <= score + n * 2.0 ** -24 + 2.0 ** -23 * (abs(rl) + e)


def rows_with_a_sink(tag, n, d, at, nats, v_scale):
    """q, k, v of which key `at` scores about `nats` more than an average key and has zero values."""
    q64 = synth.widen(synth.tensor(tag + "/q", (1, 1, d), "bf16"), "bf16")
    k64 = synth.widen(synth.tensor(tag + "/k", (n, 1, d), "bf16"), "bf16")
    v64 = synth.widen(synth.tensor(tag + "/v", (n, 1, d), "bf16"), "bf16") * v_scale
    k64[at, 0] = q64[0, 0] * (nats * math.sqrt(d) / (q64[0, 0] @ q64[0, 0]))
    v64[at] = 0
    return q64, synth.to_storage(k64, "bf16"), synth.to_storage(v64, "bf16")


@pytest.mark.parametrize("v_exp", [0, -6, -14, -16, -18, -40])
@pytest.mark.parametrize("nats", [0, 8, 10, 12, 30])
@pytest.mark.parametrize("n,at,d,wide", [(64, 0, 64, None), (64, 37, 32, None), (700, 699, 128, None), (5000, 0, 64, 1000)])
def test_zero_value_rows_do_not_hide_the_others(n, at, d, wide, nats, v_exp):
    """A key without values (an attention sink, padding) is stored with scale 2^0: whatever its score and the size of the other
    values, the others keep their precision."""
    G.require_gpu()
    q64, k, v = rows_with_a_sink(f"sink/{n}/{d}", n, d, at, nats, 2.0 ** v_exp)
    c = appended("sink", k, v, table_pages=wide)
    o, lse = attend(c, synth.to_storage(q64, "bf16"), 1 / math.sqrt(d), 1)
    check_closely(c, q64, o, lse, 1 / math.sqrt(d))


@pytest.mark.parametrize("d", [16, 64, 128])
def test_only_zero_values(d):
    G.require_gpu()
    q64, k, v = rows_with_a_sink("nothing", 300, d, 0, 3, 0.0)
    c = appended("nothing", k, v)
    o, lse = attend(c, synth.to_storage(q64, "bf16"), 1 / math.sqrt(d), 1)
    assert not G.to_f64(o).any()
    check_closely(c, q64, o, lse, 1 / math.sqrt(d))
