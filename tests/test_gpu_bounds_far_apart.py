"""Bounds of channels whose keys are far smaller than the page's largest: still the next code below and above, however far apart
they are.  Exactly the float64 oracle's."""
import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.paged import Cache
from tests.test_gpu_select import cache_of, check_bounds, make_bounds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [8, 40, 64, 128])
@pytest.mark.parametrize("large,small", [(2.0 ** 27, 2.0 ** -126), (2.0 ** 120, 2.0 ** -40), (2.0 ** 100, 2.0 ** -133), (3.0, 2.0 ** -133)])
def test_bfloat16_keys(large, small, d):
    """One large key a page and head; the other channels' keys all small, of one sign or both, or zero."""
    G.require_gpu()
    c = Cache("far/bf16", [37, 150, 1], 16, 2, d, "bf16")
    kind = np.arange(d) % 4
    sign = np.where(synth.counter_u16("far/bf16/sign", (c.pages, 2, 16, d)) % 2, -1.0, 1.0)
    sign[..., kind == 0] = -1.0
    sign[..., kind == 1] = 1.0
    rows = sign * small
    rows[..., kind == 3] = -0.0
    rows[:, :, 0, d - 1] = large
    x = synth.to_storage(rows, "bf16")
    c.dev["k"].copy_(G.to_device(x, "bf16"))
    c.host["k"] = synth.widen(x, "bf16")
    check_bounds(c, *make_bounds(c))
    binding.fa2_device_status()


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("large,small", [(200, 40), (247, 67), (140, 4)])
def test_codes(large, small, d, form):
    """Half of the channels are zero in the row of the large power of two."""
    torch = G.require_gpu()
    c = cache_of(form, "far/codes", [37, 150, 1], 16, 2, d, stale=False)
    exps = c.exps()["k_exp"]
    byte = np.full(tuple(exps.shape), small, dtype=np.uint8)
    byte[:, :, 0] = large
    exps.copy_(torch.from_numpy(byte))
    if form == "e4m3":
        codes = c.dev["k"].view(torch.uint8).cpu().numpy().copy()
        codes[:, :, 0, : d // 2] = 0
        codes[:, :, 1:, : d // 4] |= 0x80
        c.dev["k"].view(torch.uint8).copy_(torch.from_numpy(codes))
        k = S.row_values(codes, 127) * 2.0 ** (byte[..., None] - 127.0)
    else:
        codes = c.codes["k"]
        codes[:, :, 0, : d // 2] = 0
        codes[:, :, 1:, : d // 4] |= 8
        c.dev["k"].copy_(torch.from_numpy(S.pack4(codes)))
        k = S.row_values4(codes, c.scale["k"].view(torch.uint8).cpu().numpy(), byte)
    c.host["k"] = np.where(np.abs(k) >= 2.0 ** 128, np.copysign(np.inf, k), k)
    check_bounds(c, *make_bounds(c))
    binding.fa2_device_status()
