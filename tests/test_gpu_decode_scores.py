"""Scores at the ends of their range, in the attention of one new token: against the float64 oracle."""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from tests import gpu_util as G
from tests.paged import Cache
from tests.test_gpu_decode import workspace
from tests.test_gpu_decode_e4m3 import appended, attend, check_closely

pytestmark = pytest.mark.gpu


def test_scores_a_step_apart_at_2_27():
    """fp16 keys whose products with q are 2^27 + 16 j, float32's steps there, j = 1 .. 4 for a quarter of the keys each: in blocks
    of 64 keys that four warps take in turn, each warp meets all four.  The last quarter takes all, and no weight may leave
    half's range on the way."""
    torch = G.require_gpu()
    n, hkv, d = 1024, 304, 32
    c = Cache("scores/steps", [n], 64, hkv, d, "f16")
    q64, k64 = np.zeros((1, hkv, d)), np.zeros((c.pages, hkv, 64, d))
    q64[..., :9] = 4096.0
    q64[..., 9] = 1.0
    for block in range(16):
        row = np.zeros(d)
        row[:8], row[9] = 4096.0, 16.0 * (1 + block // 4)  # 2^27 and the step
        k64[c.table[0, block], :] = row
    c.host["k"] = k64
    c.dev["k"] = G.to_device(synth.to_storage(k64, "f16"), "f16")
    o, lse = G.empty((1, hkv, d), "f16"), torch.empty(1, hkv, device="cuda")
    q = G.to_device(synth.to_storage(q64, "f16"), "f16")
    for scale in (0.6931472, 0.6931471, 1.3862944):
        o.fill_(float("nan"))
        binding.fa2_decode(q, *c.pools(), o, lse, c.table_dev, c.lens_dev, workspace(1, hkv, hkv, d), scale)
        binding.fa2_device_status()
        got, last = G.to_f64(o)[0], c.rows("v", 0)[0][768:]
        assert np.isfinite(got).all() and torch.isfinite(lse).all()
        assert np.all(np.abs(got - last.mean(0)) <= (2 * 2.0 ** -11 + 512 * 2.0 ** -24) * np.abs(last).max(0))  # weights, output; sums


@pytest.mark.parametrize("dtype,e4m3", [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)])
@pytest.mark.parametrize("d,group", [(32, 1), (64, 16), (128, 4), (128, 12), (80, 8)])
@pytest.mark.parametrize("n,wide", [(16, None), (40, None), (200, None), (3000, 1000)])
def test_weights_keep_more_than_16_bits(n, wide, d, group, dtype, e4m3):
    """Scores so small that a weight rounded to 16 bits alone would be the largest error by far."""
    G.require_gpu()
    c = Cache(f"scores/weights/{n}", [n], 16, 1, d, dtype, e4m3, table_pages=wide)
    q = synth.tensor("scores/weights/q", (1, group, d), dtype, scale=2.0 ** -6)
    o, lse = attend(c, q, 1 / math.sqrt(d), group)
    check_closely(c, synth.widen(q, dtype), o, lse, 1 / math.sqrt(d), group)


@pytest.mark.parametrize("q_exp,k_exp", [(-118, 118), (-60, 60), (-100, 105), (60, -60), (90, -60), (20, 0), (-130, 100)])
@pytest.mark.parametrize("d,wide", [(64, None), (128, 500)])
def test_small_queries_and_large_keys(q_exp, k_exp, d, wide):
    """bf16 rows whose sizes make up for one another in an 8-bit cache: neither half of a score's scale may overflow alone."""
    G.require_gpu()
    n = 300
    q64 = synth.widen(synth.tensor("scores/small/q", (1, 1, d), "bf16"), "bf16") * 2.0 ** q_exp
    k64 = synth.widen(synth.tensor("scores/small/k", (n, 1, d), "bf16"), "bf16") * 2.0 ** k_exp
    v = synth.tensor("scores/small/v", (n, 1, d), "bf16")
    q = synth.to_storage(q64, "bf16")
    c = appended("scores/small", synth.to_storage(k64, "bf16"), v, table_pages=wide)
    o, lse = attend(c, q, 1 / math.sqrt(d), 1)
    check_closely(c, synth.widen(q, "bf16"), o, lse, 1 / math.sqrt(d))


def test_large_queries_beside_large_keys_at_right_angles():
    """Products of exactly 0 stay 0 whatever the scales."""
    G.require_gpu()
    n, d = 100, 32
    q64, k64 = np.zeros((1, 1, d)), np.zeros((n, 1, d))
    q64[..., : d // 2], k64[..., d // 2:] = 2.0 ** 100, 2.0 ** 110
    q = synth.to_storage(q64, "bf16")
    c = appended("scores/angles", synth.to_storage(k64, "bf16"), synth.tensor("scores/angles/v", (n, 1, d), "bf16"))
    o, lse = attend(c, q, 1 / math.sqrt(d), 1)
    check_closely(c, q64, o, lse, 1 / math.sqrt(d))
