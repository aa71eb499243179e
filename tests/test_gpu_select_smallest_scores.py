"""Selection by the smallest scores there are: bytes from 67 on and queries down to 2^-60 select as exact numbers do."""
import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from tests import gpu_util as G
from tests.paged import Cache
from tests.test_gpu_select import check_selection, select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,power", [("bf16", -60), ("bf16", -54), ("f16", -24)])
def test_smallest_powers_of_two(dtype, power):
    torch = G.require_gpu()
    c = Cache("smallest/scores", [3200, 1605], 16, 2, 64, dtype)
    codes = np.sort((synth.counter_u16("smallest/scores/bounds", (c.pages, 2, 2, 64)) % 9).astype(np.int64) - 4, axis=2)
    byte = (67 + synth.counter_u16("smallest/scores/exp", (c.pages, 2)) % 3).astype(np.uint8)
    ints = (synth.counter_u16("smallest/scores/q", (2, 6, 64)) % 5).astype(np.float64) - 2
    x = synth.to_storage(ints * 2.0 ** power, dtype)
    q64 = synth.widen(x, dtype)
    assert np.any(q64) and np.all(np.abs(q64) <= 127 * 2.0 ** power)
    for budget in (20, 150):
        table, lens = select(c, G.to_device(x, dtype), torch.from_numpy(codes.astype(np.int8)).cuda(), torch.from_numpy(byte).cuda(), budget, 0, 1)
        check_selection(c, q64, codes, byte, table, lens, budget, 0, 1)
    binding.fa2_device_status()
