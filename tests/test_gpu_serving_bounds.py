"""Each step of a generation against the cache as it stands: the stored rows against the projections, the attention against the rows.

Tighter than an end-to-end comparison, in which the rounding of the stored rows covers everything else.  Stored rows: a rotated
element is off by 5 u (|x1| + |x2|) m and its rounding to bfloat16, u = 2^-24; an e4m3 code by half a step, 2^-4 of itself or
2^-10 of the row's scale 2^e, and 224 2^e is below the row's largest magnitude.  Attention: the bound of test_gpu_decode.
"""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.test_gpu_decode import check
from tests.test_gpu_serving import D, GROUP, HEADS, HKV, Server

pytestmark = pytest.mark.gpu


def rows_held(c):
    """The cache's pages as they are on the device now, in float64."""
    import torch
    for side in "kv":
        dev = c.dev[side].contiguous()
        if c.e4m3:
            exps = c.exp[side].cpu().numpy()[..., None].astype(np.float64)
            c.host[side] = S.e4m3_values()[dev.view(torch.uint8).cpu().numpy()] * 2.0 ** (exps - 127)
        else:
            c.host[side] = G.to_f64(dev)


@pytest.mark.parametrize("e4m3", [False, True])
def test_every_step_follows_from_the_rows_it_holds(e4m3):
    torch = G.require_gpu()
    s = Server([33, 1, 64, 17], 12, e4m3)
    s.prefill()
    for i in range(s.steps):
        s.lens += 1
        rows = G.to_device(s.new_rows(i), "bf16")
        s.step(rows)
        binding.fa2_device_status()
        rows_held(s.cache)
        s.cache.lens = s.lens.tolist()
        check(s.cache, G.to_f64(rows[:, :HEADS]), s.o, s.lse, GROUP, 1 / math.sqrt(D))
        for b, x in enumerate(s.qkv):
            n = s.cache.lens[b]
            w = synth.widen(x[:n], "bf16")
            k = w[:, HEADS:HEADS + HKV]
            turned = S.rope(k.swapaxes(0, 1)[None], np.arange(n)[None], s.freq64, False, s.magnitude)[0].swapaxes(0, 1)
            pair = np.abs(k[..., : D // 2]) + np.abs(k[..., D // 2:])
            off = 5 * 2.0 ** -24 * s.magnitude * np.concatenate([pair, pair], -1)
            off = off + 2.0 ** -8 * (np.abs(turned) + off)
            for side, want, bound in (("k", turned, off), ("v", w[:, HEADS + HKV:], 0.0)):
                got, held = s.cache.rows(side, b)
                assert held.all()
                if e4m3:
                    size = np.abs(want) + bound
                    bound = bound + np.maximum(2.0 ** -4 * size, 2.0 ** -10 / 224 * size.max(-1, keepdims=True))
                assert np.all(np.abs(got - want) <= bound), f"step {i}, sequence {b}: {side}"
