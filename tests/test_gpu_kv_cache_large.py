"""Calls on so many tokens that a warp takes several rounds of them: bit for bit what many calls on few tokens do, which the
oracle's tests hold."""
import pytest

from attention_fa2_forward_02_gb300 import binding
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

# tokens past 152 * 8 blocks of 16-bit rows, 152 * 32 of e4m3 ones, of few heads; and whole tokens of more heads
CASES = [(False, 1, 64, 41003), (False, 1, 32, 81003), (False, 2, 32, 41003), (True, 1, 128, 158001), (True, 2, 64, 158001),
         (True, 1, 64, 315001), (False, 8, 128, 21003), (True, 8, 128, 21003)]


def random_bits(shape, dtype, seed):
    """Every bit pattern: infinities, NaN and subnormals among them."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randint(-32768, 32768, shape, generator=gen, device="cuda", dtype=torch.int16).view(dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("e4m3,hkv,d,tokens", CASES)
def test_one_large_call_and_many_small_ones(e4m3, hkv, d, tokens, dtype):
    torch = G.require_gpu()
    dt = getattr(torch, G.TORCH_DTYPE_NAMES[dtype])
    page = 16
    wide = -(-tokens // page)
    table = torch.randperm(wide, device="cuda").int().view(1, wide)
    rows = random_bits((tokens, 2 * hkv, d), dt, tokens)
    pools = []
    for step in (tokens, 2999):
        pages = [torch.zeros(wide, hkv, page, d, device="cuda", dtype=torch.uint8 if e4m3 else dt) for _ in "kv"]
        typed = [p.view(torch.float8_e4m3fn) if e4m3 else p for p in pages]
        exps = {f"{s}_exp": torch.zeros(wide, hkv, page, device="cuda", dtype=torch.uint8) for s in "kv"} if e4m3 else {}
        for at in range(0, tokens, step):
            end = min(at + step, tokens)
            lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([end], [0, end - at]))
            binding.fa2_kv_append(*typed, rows[at:end, :hkv], rows[at:end, hkv:], table, lens, cu_new=cu, **exps)
        out = [torch.zeros(1, hkv, tokens, d, device="cuda", dtype=dt) for _ in "kv"]
        lens = torch.tensor([tokens], dtype=torch.int32, device="cuda")
        if step == tokens:
            binding.fa2_kv_read(*typed, *out, table, lens, **exps)
        else:  # a table's part is a cache of its own
            for at in range(0, tokens, 3008):
                end = min(at + 3008, tokens)
                part = [torch.zeros(1, hkv, end - at, d, device="cuda", dtype=dt) for _ in "kv"]
                n = torch.tensor([end - at], dtype=torch.int32, device="cuda")
                binding.fa2_kv_read(*typed, *part, table[:, at // page:].contiguous(), n, **exps)
                for o, p in zip(out, part):
                    o[:, :, at:end] = p
        binding.fa2_device_status()
        pools.append([x.view(torch.uint8) for x in (*pages, *exps.values(), *out)])
    for a, b in zip(*pools):
        assert torch.equal(a, b)
