"""Rotary positions on the GPU against the float64 oracle.

Tolerance, from the arithmetic: the angle's fraction of a turn is rounded to float32 (2^-24 of an angle of at most pi:
2^-22.3), its sine and cosine and their product with the magnitude to float32 (2^-23 together), and each of the two
products and their sum to float32 (3 2^-24), all relative to m (|x1| + |x2|): below 2^-21 of it. For 16-bit types the sine
and cosine are the special function unit's, off by up to 2^-20.9 between -pi and pi: 2^-21 + 2^-20.9, below 2^-19.9 in
all. The result is then rounded to the storage type, half a step of it (u |ref|, or half its smallest subnormal step).
"""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.tolerance import UNIT_ROUNDOFF

pytestmark = pytest.mark.gpu

U = {**UNIT_ROUNDOFF, "f32": 2.0 ** -24}
TURN = {"bf16": 2.0 ** -19.9, "f16": 2.0 ** -19.9, "f32": 2.0 ** -21}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}


def check(got, ref, x, rot, interleaved, magnitude, dtype, what):
    r = rot // 2
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, r), slice(r, rot))
    size = np.zeros_like(ref)
    size[..., one] = size[..., two] = abs(magnitude) * (np.abs(x[..., one]) + np.abs(x[..., two]))
    bound = U[dtype] * np.abs(ref) + (1 + U[dtype]) * TURN[dtype] * size + TINY[dtype]
    bound[..., rot:] = 0
    over = np.abs(got - ref) > bound
    assert np.all(np.isfinite(got)) and not over.any(), f"{what}: {int(over.sum())} element(s) off, worst {np.max(np.abs(got - ref) - bound):.3e}"


def frequencies(rot):
    return 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)


def run(b, h, n, d, rot, interleaved, dtype, order, backward, in_place, pos, magnitude=1.0, freq=None):
    torch = G.require_gpu()
    freq = frequencies(rot) if freq is None else freq
    tag = f"rope/{b}/{h}/{n}/{d}"
    shape = (b, h, n, d) if order == "bhnd" else (b, n, h, d)
    x = synth.tensor(tag, shape, dtype)
    xg = G.guarded(shape, dtype)
    xg.t.copy_(G.to_device(x, dtype))
    yg = xg if in_place else G.guarded(shape, dtype)
    view = lambda t: t if order == "bhnd" else t.transpose(1, 2)  # noqa: E731
    x64 = synth.widen(x, dtype)
    x64 = x64 if order == "bhnd" else x64.swapaxes(1, 2)
    f = torch.from_numpy(freq).cuda()
    p = None if pos is None else torch.from_numpy(np.ascontiguousarray(pos, dtype=np.int32)).cuda()
    call = binding.fa2_rope_backward if backward else binding.fa2_rope
    call(view(xg.t), view(yg.t), f, positions=p, interleaved=interleaved, magnitude=magnitude)
    binding.fa2_device_status()
    full = np.broadcast_to(np.arange(n) if pos is None else pos, (b, n))
    ref = S.rope(x64, full, freq, interleaved, magnitude, backward)
    check(G.to_f64(view(yg.t)), ref, x64, rot, interleaved, magnitude, dtype, tag)
    xg.assert_intact("x")
    yg.assert_intact("y")


SIZES = [
    # b, h, n, d, rot: one token; every vector width; parts of the head; odd sizes; more pairs than threads
    (1, 1, 1, 128, 128), (2, 3, 5, 64, 64), (1, 40, 7, 128, 128), (2, 5, 33, 128, 64), (3, 2, 17, 96, 32), (1, 7, 9, 80, 40),
    (1, 3, 11, 80, 80), (2, 2, 13, 64, 18), (1, 4, 6, 7, 4), (1, 2, 3, 5, 2), (2, 1, 4, 1, 0), (1, 2, 5, 576, 576), (1, 1, 3, 1024, 1024),
    (1, 2, 300, 32, 32), (5, 3, 2, 24, 8),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("b,h,n,d,rot", [s for s in SIZES if s[4]])
def test_sizes(b, h, n, d, rot, dtype, interleaved):
    rng = np.random.default_rng(b + h + n + d)
    pos = rng.integers(0, 5000, (b, n))
    run(b, h, n, d, rot, interleaved, dtype, "bnhd" if n % 2 else "bhnd", False, False, pos, 1.2)
    run(b, h, n, d, rot, interleaved, dtype, "bhnd", True, False, None)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("order", ["bhnd", "bnhd"])
def test_in_place(order, interleaved):
    run(2, 5, 37, 96, 64, interleaved, "bf16", order, False, True, None)
    run(2, 5, 37, 30, 18, interleaved, "f16", order, True, True, None)


def test_shared_positions_and_far_ones():
    """Positions shared by all entries ([N] and [1, N]), negative ones, and the largest int32: the float64 angle
    2^31 f_i has an error of 2^-22 itself, as much as float32 has here."""
    torch = G.require_gpu()
    run(3, 2, 5, 64, 64, False, "f32", "bhnd", False, False, np.array([0, 1, -1, -70000, 9]))
    run(3, 2, 5, 64, 64, True, "f32", "bhnd", False, False, np.array([[7, 1 << 20, 123456789 % (1 << 24), 3, 1 << 22]]))
    # exactly known far angles: f = 2 pi / 2^k turns position p by p / 2^k of a turn, up to f's own rounding times p
    f = np.array([2 * math.pi / 2 ** k for k in (3, 20, 30, 31)])
    pos = np.array([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1]], dtype=np.int64)
    x = torch.zeros(1, 1, 3, 8, device="cuda", dtype=torch.float32)
    x[..., :4] = 1
    y = torch.empty_like(x)
    binding.fa2_rope(x, y, torch.from_numpy(f).cuda(), positions=torch.from_numpy(pos.astype(np.int32)).cuda())
    got = G.to_f64(y)[0, 0]
    for n in range(3):
        for i, k in enumerate((3, 20, 30, 31)):
            turns = (int(pos[0, n]) % 2 ** k) / 2 ** k
            # 2^-20: the arithmetic's 2^-21 and float64's 2^-53 f |pos| <= 2 pi 2^-53 2^28
            assert abs(got[n, i] - math.cos(2 * math.pi * turns)) < 2.0 ** -20 and abs(got[n, 4 + i] - math.sin(2 * math.pi * turns)) < 2.0 ** -20


def test_large_and_zero_frequencies():
    run(1, 2, 6, 16, 16, False, "f32", "bhnd", False, False, np.arange(6)[None], freq=np.array([0.0, -0.5, 1.0, 3.0, 7.5, 100.25, 1e-30, 5e-324]))


def test_broadcast_input_and_slices():
    """A head repeated by a stride of 0; q and k as slices of one projection, written back in place."""
    torch = G.require_gpu()
    x = synth.tensor("rope/bcast", (2, 1, 9, 64), "bf16")
    xd, f = G.to_device(x, "bf16"), torch.from_numpy(frequencies(64)).cuda()
    y = G.empty((2, 4, 9, 64), "bf16")
    binding.fa2_rope(xd.expand(2, 4, 9, 64), y, f)
    x64 = np.broadcast_to(synth.widen(x, "bf16"), (2, 4, 9, 64))
    check(G.to_f64(y), S.rope(x64, np.broadcast_to(np.arange(9), (2, 9)), frequencies(64), False), x64, 64, False, 1.0, "bf16", "repeated")
    qkv = synth.tensor("rope/qkv", (2, 9, 8, 64), "bf16")  # 4 query, 2 key, 2 value heads
    t = G.to_device(qkv, "bf16")
    binding.fa2_rope(t[:, :, :6].transpose(1, 2), t[:, :, :6].transpose(1, 2), f)
    w = synth.widen(qkv, "bf16")
    ref = w.copy()
    ref[:, :, :6] = S.rope(w[:, :, :6].swapaxes(1, 2), np.broadcast_to(np.arange(9), (2, 9)), frequencies(64), False).swapaxes(1, 2)
    check(G.to_f64(t)[:, :, :6], ref[:, :, :6], w[:, :, :6], 64, False, 1.0, "bf16", "q and k")
    assert np.array_equal(G.to_f64(t)[:, :, 6:], w[:, :, 6:])


def test_many_entries_and_heads():
    """More (entry, part of the heads) pairs than a grid's second dimension holds."""
    run(70001, 1, 1, 8, 8, False, "bf16", "bhnd", False, False, None)
    run(1, 70001, 1, 8, 8, True, "bf16", "bhnd", False, False, np.array([[3]]))
    run(3, 40000, 1, 8, 4, True, "f16", "bhnd", False, False, np.array([[3], [4], [5]]))


def test_offsets_past_2_31_elements():
    torch = G.require_gpu()
    d, step = 64, (1 << 31) + 512
    buf = torch.empty(2 * step + 4096, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, 1, 2, d), (step, 2 * d, d, 1))
    x.copy_(G.to_device(synth.tensor("rope/far", (3, 1, 2, d), "bf16"), "bf16"))
    x64 = G.to_f64(x)
    binding.fa2_rope(x, x, torch.from_numpy(frequencies(d)).cuda())
    ref = S.rope(x64, np.broadcast_to(np.arange(2), (3, 2)), frequencies(d), False)
    check(G.to_f64(x), ref, x64, d, False, 1.0, "bf16", "far rows")


def test_gradient_against_differences():
    """sum(dy * rope(x)) grows by dx . e along a direction e: float32 values, the map is linear in x."""
    torch = G.require_gpu()
    shape, f = (2, 3, 11, 32), torch.from_numpy(frequencies(24)).cuda()
    x, e, dy = (G.to_device(synth.tensor(f"rope/grad/{n}", shape, "f32"), "f32") for n in "xed")
    y0, y1, dx = (torch.empty_like(x) for _ in range(3))
    for inter in (False, True):
        binding.fa2_rope(x - e, y0, f, interleaved=inter, magnitude=1.3)
        binding.fa2_rope(x + e, y1, f, interleaved=inter, magnitude=1.3)
        binding.fa2_rope_backward(dy, dx, f, interleaved=inter, magnitude=1.3)
        along = ((y1 - y0).double() * dy.double()).sum() / 2
        # each y within 2^-20 of values of size ~ 4 m: 2112 terms of at most 16 * 1.3 * 2^-20 in all directions
        assert abs(float(along - (dx.double() * e.double()).sum())) < 2112 * 16 * 1.3 * 2.0 ** -20
