"""Rotary positions where a sine or cosine is next to nothing: the angle, not a table or an approximation, decides.

The angle is a fraction of a turn, cut to 2^-32 (2 pi 2^-32 < 2^-29.3), less its nearest quarter, which is exact, so that a small
sine or cosine has small errors: with u = 2^-24, 3 u of the rest of the angle from its conversion and scaling and 1.4 u from the
sum, together below 5 u of itself.  The product with the input adds u, the other one is 0; then half a step of the result.
"""
import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding
from tests import gpu_util as G
from tests.tolerance import UNIT_ROUNDOFF

pytestmark = pytest.mark.gpu

U = {**UNIT_ROUNDOFF, "f32": 2.0 ** -24}


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("turn", [-0.25, 0.0, 0.25, 0.5, 0.75, 1.0])
@pytest.mark.parametrize("backward", [False, True])
def test_next_to_the_quarter_turns(turn, dtype, backward):
    torch = G.require_gpu()
    rot = 1024
    delta = np.concatenate([s * 2.0 ** -np.linspace(9, 18, rot // 4) for s in (1, -1)])  # of a turn
    freq = 2 * np.pi * (turn + delta)
    x = torch.zeros(1, 1, 1, rot, dtype=getattr(torch, G.TORCH_DTYPE_NAMES[dtype]), device="cuda")
    x[..., : rot // 2] = 1024.0
    y = torch.empty_like(x)
    call = binding.fa2_rope_backward if backward else binding.fa2_rope
    call(x, y, torch.from_numpy(freq).cuda(), positions=torch.ones(1, 1, dtype=torch.int32, device="cuda"))
    got = G.to_f64(y).reshape(2, rot // 2) / 1024.0
    # cos and sin of 2 pi (turn + delta) from delta alone, which float64 holds exactly
    c, s = np.cos(2 * np.pi * delta), np.sin(2 * np.pi * delta)
    quarter = int(round(turn * 4)) % 4
    cos, sin = ((c, s), (-s, c), (-c, -s), (s, -c))[quarter]
    if backward:
        sin = -sin
    for name, g, ref in (("cos", got[0], cos), ("sin", got[1], sin)):
        # 2^-51: the frequency, a double of up to 2 pi 1.002
        bound = 6 * 2.0 ** -24 * np.abs(ref) + 2 * np.pi * 2.0 ** -32 + 2.0 ** -51
        bound = bound + U[dtype] * (np.abs(ref) + bound)
        over = np.abs(g - ref) > bound
        assert not over.any(), f"{name}: {int(over.sum())} off, worst {np.max(np.abs(g - ref) / bound):.3g} times its bound"


def test_sines_and_cosines_all_around():
    """float32, (1, 0) turned: within 5 u (3.4 u of the sum, u of the product)."""
    torch = G.require_gpu()
    rot, n = 1024, 2000
    freq = 2 * np.pi * (np.arange(rot // 2) + 0.37) / (rot // 2)
    pos = np.arange(n, dtype=np.int32)
    x = torch.zeros(1, 1, n, rot, device="cuda")
    x[..., : rot // 2] = 1.0
    y = torch.empty_like(x)
    binding.fa2_rope(x, y, torch.from_numpy(freq).cuda(), positions=torch.from_numpy(pos).cuda())
    angle = pos[:, None].astype(np.float64) * freq  # up to 2^14: off by 2^-39
    got = G.to_f64(y)[0, 0]
    for g, ref in ((got[:, : rot // 2], np.cos(angle)), (got[:, rot // 2:], np.sin(angle))):
        assert np.max(np.abs(g - ref)) <= 5 * 2.0 ** -24
