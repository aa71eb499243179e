"""Which division of the work fa2_decode takes: the rule of its sizes, written out, against what the library records."""
import math

import pytest

from attention_fa2_forward_02_gb300 import binding
from tests.test_gpu_decode import run, workspace

pytestmark = pytest.mark.gpu


def ctas_per_item(batch, hkv, group, d, e4m3, room, window=0):
    """One launch of clusters, the largest of up to 8 CTAs with which all items are resident and every warp still has a block,
    where no warp can have more than 4 blocks (8 with more items than resident CTAs); else 0."""
    kernel_d = 32 if d <= 32 else 64 if d <= 64 else 128
    row_bytes = kernel_d if e4m3 else 2 * kernel_d
    block = 16 if row_bytes >= 256 else 32 if row_bytes == 128 else 64
    per_sm = 3 if (group <= 8 and row_bytes < 256) or (e4m3 and kernel_d == 32) else 2
    items, resident = batch * hkv * -(-group // (8 if group <= 8 else 16)), 152 * per_sm
    keys = min(room, window + 15) if window else room
    blocks, ctas = -(-keys // block), 1
    while ctas < 8 and 2 * ctas * items <= resident and blocks > 4 * ctas:
        ctas *= 2
    return ctas if blocks <= 4 * ctas * (8 if items > resident else 4) else 0


CASES = [  # batch, hkv, group, table width in pages of 16
    (1, 1, 1, 17), (1, 1, 1, 200), (1, 8, 4, 17), (1, 8, 4, 63), (3, 2, 16, 17), (9, 8, 3, 17), (70, 8, 2, 17), (70, 8, 2, 40),
    (1, 8, 4, 2000), (70, 8, 2, 2000), (2, 304, 1, 60), (20, 4, 20, 17),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [32, 64, 80, 128])
@pytest.mark.parametrize("batch,hkv,group,wide", CASES)
def test_short_contexts_take_clusters(batch, hkv, group, wide, d, e4m3):
    lens = [(37 * i * i + 5 * i) % 260 for i in range(batch)]
    lens[0] = 259
    for window in (0, 77):
        run("paths/short", lens, 16, hkv, group, d, "bf16", e4m3, window=window, table_pages=wide, rows=[0])
        assert binding.fa2_last_decode_info() == ctas_per_item(batch, hkv, group, d, e4m3, 16 * wide, window)


def test_every_division_is_among_the_cases():
    got = {ctas_per_item(*c[:3], d, e, 16 * c[3], w) for c in CASES for d in (32, 64, 80, 128) for e in (False, True) for w in (0, 77)}
    assert got == {0, 1, 2, 4, 8}


@pytest.mark.parametrize("window", [3000, 4000, 1 << 40, 2 ** 63 - 16, 2 ** 63 - 15, 2 ** 63 - 1])
def test_windows_as_wide_as_the_table_and_wider(window):
    """They leave all keys: the division and the bits of a call without one."""
    import torch
    c, q, o, lse = run("paths/wide", [2900, 700], 16, 2, 4, 128, table_pages=188)
    assert binding.fa2_last_decode_info() == 0
    o2, l2 = torch.empty_like(o), torch.empty_like(lse)
    binding.fa2_decode(q, *c.pools(), o2, l2, c.table_dev, c.lens_dev, workspace(2, 8, 2, 128), 1 / math.sqrt(128), window=window)
    assert binding.fa2_last_decode_info() == 0
    assert torch.equal(o, o2) and torch.equal(lse, l2)
