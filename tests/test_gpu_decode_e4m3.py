"""Value rows of an 8-bit cache whose scales lie far apart, in the attention of one new token: against the float64 oracle."""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.paged import Cache
from tests.test_gpu_decode import check, workspace

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
