"""Pins of oracle/serving.py, and the host-side frequencies of rotary positions (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding
from attention_fa2_forward_02_gb300 import build as build_mod
from oracle import attention as A
from oracle import serving as S


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return binding.library()


# ---------------------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_the_written_out_formula(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 3, 4, 10))
    f, pos, mag = np.array([0.7, 0.01, 3.0]), np.array([[0, 5, -2, 100], [1, 1, 7, 3]]), 1.25
    y = S.rope(x, pos, f, interleaved, mag)
    for b in range(2):
        for n in range(4):
            for i in range(3):
                one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + 3)
                c, s = math.cos(pos[b, n] * f[i]), math.sin(pos[b, n] * f[i])
                assert np.allclose(y[b, :, n, one], mag * (x[b, :, n, one] * c - x[b, :, n, two] * s), atol=1e-13)
                assert np.allclose(y[b, :, n, two], mag * (x[b, :, n, two] * c + x[b, :, n, one] * s), atol=1e-13)
    assert np.array_equal(y[..., 6:], x[..., 6:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_backward_is_the_gradient(interleaved):
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((2, 1, 2, 3, 8))
    f, pos = np.array([0.9, 0.05]), np.array([[3, 400, 9]])
    dx = S.rope(dy, pos, f, interleaved, 1.1, backward=True)
    loss = lambda z: float(np.sum(S.rope(z, pos, f, interleaved, 1.1) * dy))  # noqa: E731
    for i in np.ndindex(x.shape):
        step = np.zeros_like(x)
        step[i] = 1e-4
        assert abs((loss(x + step) - loss(x - step)) / 2e-4 - dx[i]) < 1e-8


def test_rope_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((2, 1, 1, 1, 16))
    f = 10000.0 ** (-np.arange(8) / 8)
    dot = lambda a, b: float(np.sum(S.rope(q, [[a]], f, True) * S.rope(k, [[b]], f, True)))  # noqa: E731
    assert abs(dot(17, 5) - dot(112, 100)) < 1e-12


def _freq(lib, rot, base, kind, factor=1.0, length=0.0, low=1.0, high=32.0):
    out, mag = (ctypes.c_double * (rot // 2))(), ctypes.c_float()
    st = lib.fa2_rope_frequencies(out, ctypes.byref(mag), rot, base, kind, factor, length, low, high)
    return st, np.array(out[:]), mag.value


def test_frequencies(lib):
    i = np.arange(32)
    plain = 500000.0 ** (-2 * i / 64)
    assert np.allclose(_freq(lib, 64, 500000.0, 0)[1], plain, rtol=1e-14)
    assert np.allclose(_freq(lib, 64, 500000.0, 1, 4.0)[1], plain / 4, rtol=1e-14)
    assert np.allclose(_freq(lib, 64, 10000.0, 2, 4.0)[1], (10000.0 * 4 ** (64 / 62)) ** (-2 * i / 64), rtol=1e-13)
    # mixed by turns over the original length: fast ones as they are, slow ones divided, between them a blend
    st, f, mag = _freq(lib, 64, 500000.0, 3, 8.0, 8192.0, 1.0, 4.0)
    turns = 8192.0 * plain / (2 * math.pi)
    assert st == 0 and mag == 1.0
    assert np.allclose(f[turns >= 4], plain[turns >= 4], rtol=1e-14)
    assert np.allclose(f[turns <= 1], plain[turns <= 1] / 8, rtol=1e-14)
    between = (turns > 1) & (turns < 4)
    assert between.any()
    w = (turns[between] - 1) / 3
    assert np.allclose(f[between], plain[between] * (w + (1 - w) / 8), rtol=1e-12)
    # mixed along the index
    st, f, mag = _freq(lib, 64, 10000.0, 4, 16.0, 4096.0, 1.0, 32.0)
    plain = 10000.0 ** (-2 * i / 64)
    at = lambda t: 64 * math.log(4096 / (t * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    a, b = math.floor(at(32)), math.ceil(at(1))
    w = 1 - np.clip((i - a) / (b - a), 0, 1)
    assert st == 0 and abs(mag - (0.1 * math.log(16) + 1)) < 1e-6
    assert np.allclose(f, plain * (w + (1 - w) / 16), rtol=1e-12)
    f2, mag2 = binding.fa2_rope_frequencies(64, 10000.0, "ramp", 16.0, 4096.0)
    assert np.array_equal(f2.numpy(), f) and mag2 == mag


def test_frequencies_refusals(lib):
    out = (ctypes.c_double * 32)()
    call = lambda *a: lib.fa2_rope_frequencies(*a)  # noqa: E731
    assert call(None, None, 64, 1e4, 0, 1.0, 0.0, 1.0, 32.0) == 1
    assert call(out, None, 63, 1e4, 0, 1.0, 0.0, 1.0, 32.0) == 1
    assert call(out, None, 0, 1e4, 0, 1.0, 0.0, 1.0, 32.0) == 1
    assert call(out, None, 64, -1.0, 0, 1.0, 0.0, 1.0, 32.0) == 1
    assert call(out, None, 64, 1e4, 5, 1.0, 0.0, 1.0, 32.0) == 1
    assert call(out, None, 64, 1e4, 1, 0.5, 0.0, 1.0, 32.0) == 1
    assert call(out, None, 64, 1e4, 3, 2.0, 0.0, 1.0, 32.0) == 1
    assert call(out, None, 64, 1e4, 3, 2.0, 100.0, 4.0, 4.0) == 1
    assert call(out, None, 2, 1e4, 2, 2.0, 0.0, 1.0, 32.0) == 1
    assert call(out, None, 64, 1.0, 4, 2.0, 100.0, 1.0, 32.0) == 1
    assert call(out, None, 64, 1e4, 0, math.nan, 0.0, 1.0, 32.0) == 0  # unused there
    with pytest.raises(ValueError):
        binding.fa2_rope_frequencies(64, scaling="other")
    with pytest.raises(binding.Fa2Error):
        binding.fa2_rope_frequencies(-2)


# ---------------------------------------------------------------------------- the 8-bit rows
def test_e4m3_values():
    v = S.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7E] == 448.0
    assert np.isnan(v[0x7F]) and v[0x80 | 0x38] == -1.0 and np.all(np.diff(v[:127]) > 0)


def test_quantise_row():
    codes, byte = S.quantise_row([448.0, 1.0, 0.0, -224.0])
    assert byte == 127 and list(S.row_values(codes, byte)) == [448.0, 1.0, 0.0, -224.0]
    assert S.quantise_row([449.0, 1.0])[1] == 128 and S.quantise_row([224.0])[1] == 126
    assert S.quantise_row([0.0, -0.0])[1] == 127
    assert S.quantise_row([1e-300])[1] == 127 + S.MIN_EXP
    codes, byte = S.quantise_row([np.inf, -np.inf, np.nan, 1.0])
    got = S.row_values(codes, byte)
    assert byte == 127 - 8 and got[0] == 448 * 2.0 ** -8 and got[1] == -got[0] and np.isnan(got[2]) and got[3] == 1.0
    # every value within half a step of 4 bits, or of the smallest step
    rng = np.random.default_rng(4)
    x = rng.standard_normal(200) * np.exp(rng.standard_normal(200))
    codes, byte = S.quantise_row(x)
    assert np.all(np.abs(S.row_values(codes, byte) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (byte - 127 - 10)))
    # ties to the even fraction
    assert S.row_values(*S.quantise_row([448.0, 17.0, 19.0])).tolist() == [448.0, 16.0, 20.0]


# ---------------------------------------------------------------------------- cache and attention
def test_append_and_rows():
    table, lens, cu = np.array([[2, 0, -1], [3, 9, 1]]), [5, 7], [0, 2, 5]
    got = S.append_slots(table, lens, cu, 3, 4)
    # sequence 0: positions 3, 4 -> page 0 slots 0, 1; sequence 1: positions 4, 5 in page 9 (outside), 6 in page 1
    assert got == [(0, 0, 0), (1, 0, 1), (4, 1, 0)]
    assert S.append_slots(table, [1, 0], None, 3, 4) == [(0, 2, 0)]
    assert S.append_slots(table, [1, 99], [0, 2, 3], 3, 4) == [(1, 2, 0)]
    pages = np.arange(4 * 1 * 3 * 1, dtype=float).reshape(4, 1, 3, 1)
    rows, held = S.rows_of(pages, table[1], 7, 3, 4)
    assert rows[:, 0, 0].tolist() == [9, 10, 11, 0, 0, 0, 3] and held.tolist() == [True] * 3 + [False] * 3 + [True]


def test_decode_row_is_the_forward():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal(8), rng.standard_normal((20, 8)), rng.standard_normal((20, 8))
    o, lse, w, e = S.decode_row(q, k, v, 0.3)
    ro, rl = A.forward(q[None, None], k[None], v[None], 0.3)
    assert np.allclose(o, ro[0, 0], atol=1e-14) and abs(lse - rl[0, 0]) < 1e-13 and np.all(w >= np.abs(o)) and e > 0
    live = np.arange(20) >= 15
    assert np.allclose(S.decode_row(q, k, v, 0.3, live)[0], S.decode_row(q, k[15:], v[15:], 0.3)[0])
    o, lse, _, _ = S.decode_row(q, k, v, 0.3, np.zeros(20, bool))
    assert not o.any() and lse == -np.inf
