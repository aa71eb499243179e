"""Bounds of pages with rows of the smallest powers of two that a byte names, far below the others' in their page: a key that is not
zero lies between its bounds however small it is.  Exactly the float64 oracle's."""
import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.test_gpu_select import cache_of, check_bounds, make_bounds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("others", [9, 15, 20, 60, 127])
def test_smallest_codes_of_the_smallest_bytes(others, d, form):
    torch = G.require_gpu()
    c = cache_of(form, "smallest", [200, 31, 5], 16, 2, d, stale=False)
    exps = c.exps()["k_exp"]
    byte = 1 + synth.counter_u16(f"smallest/{others}", tuple(exps.shape)).astype(np.int64) % 5
    byte[:, :, ::4] = others
    exps.copy_(torch.from_numpy(byte.astype(np.uint8)))
    # but in the rows of the smallest bytes most channels are 0, and there the smallest code of either sign
    small = byte < 6
    if form == "e4m3":
        codes = c.dev["k"].view(torch.uint8).cpu().numpy().copy()
        codes[~small, : d // 2] = 0
        codes[small, : d // 2] = np.where(np.arange(d // 2) % 2, 0x81, 1)
        c.dev["k"].view(torch.uint8).copy_(torch.from_numpy(codes))
        c.host["k"] = S.row_values(codes, 127) * 2.0 ** (byte - 127.0)[..., None]
    else:
        codes, scales = c.codes["k"], c.scale["k"].view(torch.uint8).cpu().numpy()
        codes[~small, : d // 2] = 0
        codes[small, : d // 2] = np.where(np.arange(d // 2) % 2, 9, 1)
        scales[small, : d // 32] = 1  # 2^-9
        c.dev["k"].copy_(torch.from_numpy(S.pack4(codes)))
        c.scale["k"].view(torch.uint8).copy_(torch.from_numpy(scales))
        c.host["k"] = S.row_values4(codes, scales, byte)
    check_bounds(c, *make_bounds(c))
    binding.fa2_device_status()
