"""Value rows of zeros in a 4-bit cache, whose power of two lies far above the others', whatever a kernel before left in shared memory.

The tolerance is that of test_gpu_decode_e2m1.py's test of such rows: weights within 2^-11 each, sums of n in float32, and half's
smallest step beside the largest weight, which is a row's that is not all zeros: each |v_j| counts with no more than 2^-25 of it."""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.paged4 import Cache4
from tests.test_gpu_decode import workspace

pytestmark = pytest.mark.gpu

GROUP = 2


def cache_with_zero_rows(lens, d, table_pages):
    import torch
    c = Cache4(f"zeros/{d}", lens, 16, 1, d, table_pages=table_pages)
    slots = np.arange(c.pages * 16).reshape(c.pages, 1, 16)
    for side, low, high in (("k", 100, 120), ("v", 70, 100)):
        e = np.where(slots % 5 == 0, high, low).astype(np.uint8)
        if side == "v":
            c.codes[side][slots % 3 == 0] = 0
            e[slots % 3 == 0] = 127
        c.host[side] = S.row_values4(c.codes[side], c.scale[side].view(torch.uint8).cpu().numpy(), e)
        c.dev[side].copy_(torch.from_numpy(S.pack4(c.codes[side])))
        c.exp[side].copy_(torch.from_numpy(e))
    return c


def leave_codes_in_shared_memory():
    """A decode whose CTAs, on every SM, fill their rings with rows of 128 codes that are not zeros."""
    import torch
    pages, hkv, page, d = 200, 8, 16, 128
    pools = [torch.full((pages, hkv, page, d // 2), 0x33, dtype=torch.uint8, device="cuda") for _ in "kv"]
    form = {f"{s}_exp": torch.full((pages, hkv, page), 120, dtype=torch.uint8, device="cuda") for s in "kv"}
    form.update({f"{s}_scale": torch.full((pages, hkv, page, d // 16), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for s in "kv"})
    table = torch.arange(200, dtype=torch.int32, device="cuda").repeat(16, 1)
    lens = torch.full((16,), 3200, dtype=torch.int32, device="cuda")
    q = torch.ones(16, hkv * GROUP, d, dtype=torch.bfloat16, device="cuda")
    binding.fa2_decode(q, *pools, torch.empty_like(q), torch.empty(16, hkv * GROUP, device="cuda"), table, lens, workspace(16, hkv * GROUP, hkv, d), 0.1,
                       **form)


@pytest.mark.parametrize("table_pages", [None, 4000])  # one launch, two
@pytest.mark.parametrize("d", [128, 96, 64, 32])
def test_zero_rows_do_not_raise_the_maximum(d, table_pages):
    torch = G.require_gpu()
    lens = [300, 47, 16]
    c = cache_with_zero_rows(lens, d, table_pages)
    q = synth.tensor(f"zeros/{d}/q", (len(lens), GROUP, d), "bf16")
    dev, q64 = G.to_device(q, "bf16"), synth.widen(q, "bf16")
    results = []
    for selected in (False, True, False):
        o, lse = G.empty((len(lens), GROUP, d), "bf16"), torch.empty(len(lens), GROUP, device="cuda")
        ws = workspace(len(lens), GROUP, 1, d)
        leave_codes_in_shared_memory()
        if selected:
            table, n = c.table_dev[:, None].contiguous(), c.lens_dev[:, None].contiguous()
            binding.fa2_decode_selected(dev, *c.pools(), o, lse, table, n, ws, 0.2, **c.exps())
        else:
            binding.fa2_decode(dev, *c.pools(), o, lse, c.table_dev, c.lens_dev, ws, 0.2, **c.exps())
        binding.fa2_device_status()
        results.append((o, lse))
        for b, n in enumerate(lens):
            k, v, e_j = c.rows("k", b)[0][:, 0], c.rows("v", b)[0][:, 0], c.value_exps(b, 0)
            live = np.abs(v).sum(1) > 0
            for h in range(GROUP):
                ref, rl, w, e = S.decode_row(q64[b, h], k, v, 0.2)
                score = (d + 8) * 2.0 ** -24 * e + 2.0 ** -21
                x = 0.2 * (k @ q64[b, h]) / math.log(2) + e_j
                top = e_j[live][np.argmax(x[live])]
                bound = ((2.0 ** -11 + 2 * score + 2 * n * 2.0 ** -24) * w + 2.0 ** -8 * np.abs(ref)
                         + 2.0 ** -25 * (2.0 ** (top - e_j[live]) @ np.abs(v[live])))
                assert np.all(np.abs(G.to_f64(o)[b, h] - ref) <= bound + 1e-38), (selected, b, h)
                assert abs(float(lse[b, h]) - rl) <= score + n * 2.0 ** -24 + 2.0 ** -23 * (abs(rl) + e), (selected, b, h)
    assert torch.equal(results[0][0], results[2][0]) and torch.equal(results[0][1], results[2][1])
