"""Bounds of pages with infinities among their keys: the power of two is that of the largest finite key, wherever that lies.
Exactly the float64 oracle's."""
import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.paged import Cache
from tests.test_gpu_select import cache_of, check_bounds, make_bounds


def test_the_oracle_counts_every_finite_key():
    k = np.array([[1.0, -np.inf, 0.5], [1000.0, -300.0, 0.25], [np.inf, 2.0, np.nan]])
    codes, byte = S.page_bounds(k)
    assert byte == 127 + 3  # 1000 <= 127 * 2^3
    assert codes.tolist() == [[0, -127, 0], [127, 1, 1]]
    finite = np.where(np.isfinite(k), k, 0.0)
    assert np.all(codes[0] * 8.0 <= finite) and np.all(finite <= codes[1] * 8.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [8, 40, 64, 128])
@pytest.mark.parametrize("page", [2, 16, 64, 200])
def test_large_keys_in_a_channel_with_infinities(page, d, dtype):
    """The largest finite key of a page, far above all others, lies between infinities, or beside one; in any row."""
    G.require_gpu()
    lens = [37, 150, 1, 64, 200]
    c = Cache(f"infinities/{page}", lens, page, 3, d, dtype, stale="nan")
    rows = synth.widen(synth.tensor(f"infinities/{page}/x", (c.pages, 3, page, d), dtype), dtype)
    pick = synth.counter_u16(f"infinities/{page}/at", (c.pages, 3, 5)).astype(int)
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            p, live = c.table[b, j], min(page, n - j * page)
            for h in range(3):
                r, s, t, ch, kind = pick[p, h]
                x = rows[p, h, :live, ch % d]
                x[r % live] = 3000.0 if kind & 1 else -3000.0
                if s % live != r % live:
                    x[s % live] = np.inf
                if t % live != r % live and kind & 2:
                    x[t % live] = -np.inf
    rows[c.table[4, 0], 0] = np.inf      # nothing finite
    rows[c.table[4, 0], 1, ::2] = -np.inf
    x = synth.to_storage(rows, dtype)
    c.dev["k"].copy_(G.to_device(x, dtype))
    c.host["k"] = synth.widen(x, dtype)
    check_bounds(c, *make_bounds(c))
    binding.fa2_device_status()


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_codes_past_float32_count_as_infinite(d, form):
    """Bytes up to 253: an element of 2^128 and more is past float32, the others of its channel and page count as they are."""
    torch = G.require_gpu()
    c = cache_of(form, "infinities/codes", [200, 31, 5], 16, 2, d, stale=False)
    exps = c.exps()["k_exp"]
    for low, high in ((118, 253), (240, 253), (246, 253)):
        byte = low + synth.counter_u16(f"infinities/{low}", tuple(exps.shape)).astype(np.int64) % (high - low + 1)
        c.host["k"] = c.host["k"] * 2.0 ** (byte - exps.cpu().numpy())[..., None]
        exps.copy_(torch.from_numpy(byte.astype(np.uint8)))
        plain = c.host["k"]
        c.host["k"] = np.where(np.abs(plain) >= 2.0 ** 128, np.copysign(np.inf, plain), plain)
        assert np.isinf(c.host["k"]).any()
        check_bounds(c, *make_bounds(c))
        c.host["k"] = plain
    binding.fa2_device_status()
