"""4-bit rows into the cache's pages and back, bit for bit against the float64 oracle (a zero's sign aside)."""
import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.tolerance import UNIT_ROUNDOFF

pytestmark = pytest.mark.gpu


class Pools:
    """Pages of 4-bit rows filled with a byte pattern, scales and bytes likewise."""

    def __init__(self, pages, hkv, page, d, order="hnd", fill=0xA5):
        import torch
        self.shape, self.page, self.d, self.fill = (pages, hkv, page), page, d, fill
        base = lambda *s: torch.full(s, fill, dtype=torch.uint8, device="cuda")  # noqa: E731
        dims = (pages, hkv, page, d // 2) if order == "hnd" else (pages, page, hkv, d // 2)
        self.k, self.v = ((t if order == "hnd" else t.transpose(1, 2)) for t in (base(*dims), base(*dims)))
        self.exps = {f"{s}_exp": base(*self.shape) for s in "kv"}
        self.scales = {f"{s}_scale": base(*self.shape, d // 16).view(torch.float8_e4m3fn) for s in "kv"}

    def kw(self):
        return {**self.exps, **self.scales}

    def host(self, side):
        """(codes [pages, hkv, page, d], scale bytes, bytes)"""
        import torch
        packed = getattr(self, side).contiguous().cpu().numpy()
        codes = np.stack([packed & 15, packed >> 4], -1).reshape(*self.shape, self.d)
        return codes, self.scales[side + "_scale"].view(torch.uint8).cpu().numpy(), self.exps[side + "_exp"].cpu().numpy()


def same_codes(got, want):
    """Equal magnitudes, and signs where they are not zero."""
    assert np.array_equal(got & 7, want & 7)
    assert np.array_equal(np.where(got & 7, got, 0), np.where(want & 7, want, 0))


def rows_of(tag, shape, dtype):
    """Rows with ordinary values of growing spread, and rows of zeros, infinities, NaN, huge, tiny and in-between ones among them."""
    x = synth.tensor(tag, shape, dtype)
    w = synth.widen(x, dtype) * np.exp2(np.arange(shape[0]) % 9 - 4.0)[:, None, None]
    d = shape[-1]
    top = 60000.0 if dtype == "f16" else 2.0 ** 127
    special = [np.zeros(d), np.full(d, -0.0), np.r_[np.inf, np.ones(d - 1)], np.r_[np.full(d - 1, 0.75), -np.inf], np.r_[np.nan, np.ones(d - 1)],
               np.full(d, np.inf), np.full(d, np.nan), np.r_[top, -top, np.ones(d - 2)], np.full(d, 2.0 ** -24), np.r_[1.0, np.full(d - 1, 2.0 ** -20)],
               np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], d // 8), np.tile([-0.25, 0.75, -1.25, 1.75, -2.5, 3.5, -5.0, 6.0], d // 8) * 13 / 8]
    for i, row in enumerate(special):
        w[(5 * i) % shape[0], i % shape[1]] = row
    return synth.to_storage(w, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("order", ["hnd", "nhd"])
@pytest.mark.parametrize("hkv,page,d", [(1, 16, 32), (2, 1, 64), (3, 24, 96), (8, 16, 128), (5, 64, 64), (1, 8, 128)])
def test_append_and_read(hkv, page, d, order, dtype):
    torch = G.require_gpu()
    new, before = [7, 0, 33, 1], [5, 3, 0, 40]
    lens = [a + b for a, b in zip(new, before)]
    wide = -(-max(lens) // page)
    pages = len(lens) * wide + 2
    table = np.argsort(synth.raw_words(3, f"e2m1/{page}", 0, pages), kind="stable")[: len(lens) * wide].reshape(len(lens), wide).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) + 2  # two rows that belong to nobody
    total = int(cu[-1]) + 3
    p = Pools(pages, hkv, page, d, order)
    x = rows_of(f"e2m1/{hkv}/{page}/{d}", (total, 2 * hkv, d), dtype)
    kv = G.to_device(x, dtype)
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    binding.fa2_kv_append(p.k, p.v, kv[:, :hkv], kv[:, hkv:], dev(table), dev(lens), cu_new=dev(cu), **p.kw())
    binding.fa2_device_status()
    w = synth.widen(x, dtype)
    slots = S.append_slots(table, lens, cu, page, pages)
    assert len(slots) == sum(new)
    for side, first in (("k", 0), ("v", hkv)):
        codes, scales, bytes_ = p.host(side)
        untouched = np.ones((pages, page), dtype=bool)
        for t, pg, slot in slots:
            untouched[pg, slot] = False
            for h in range(hkv):
                c, s, e = S.quantise_row4(w[t, first + h])
                assert bytes_[pg, h, slot] == e and np.array_equal(scales[pg, h, slot], s), (t, h)
                groups = np.repeat(s != 0x7F, 16)  # a NaN's codes mean nothing
                same_codes(codes[pg, h, slot][groups], c[groups])
        rest = np.broadcast_to(untouched[:, None], p.shape)
        assert np.all(bytes_[rest] == p.fill) and np.all(scales[rest] == p.fill) and np.all(codes[rest] == np.tile([p.fill & 15, p.fill >> 4], d // 2))
    # ---- read back what was stored (the rows before, of the fill pattern, with it)
    out = [G.guarded((len(lens), hkv, max(lens) + 3, d), dtype) for _ in "kv"]
    before_read = out[0].t.clone()
    binding.fa2_kv_read(p.k, p.v, out[0].t, out[1].t, dev(table), dev(lens), **p.kw())
    binding.fa2_device_status()
    for side, o in zip("kv", out):
        o.assert_intact(side)
        codes, scales, bytes_ = p.host(side)
        got = G.to_f64(o.t)
        for b, n in enumerate(lens):
            at = [(table[b][pos // page], slice(None), pos % page) for pos in range(n)]
            ref = np.stack([S.row_values4(codes[i], scales[i], bytes_[i]) for i in at], 1) if n else np.zeros((hkv, 0, d))
            with np.errstate(over="ignore", invalid="ignore"):
                ref = ref if dtype == "bf16" else ref.astype(np.float16).astype(np.float64)
            assert np.array_equal(got[b, :, :n], ref, equal_nan=True)
        tail = o.t.view(torch.int16)
        for b, n in enumerate(lens):
            assert torch.equal(tail[b, :, n:], before_read.view(torch.int16)[b, :, n:])


@pytest.mark.parametrize("tokens,hkv,d", [(1, 1, 128), (2500, 2, 64), (900, 8, 128), (5000, 1, 32)])
def test_append_of_few_and_of_many_tokens(tokens, hkv, d):
    """Every way a call divides its rows: one sequence, all of its tokens; values within a step of what was stored."""
    torch = G.require_gpu()
    page = 32
    wide = -(-tokens // page)
    p = Pools(wide, hkv, page, d)
    x = synth.tensor(f"e2m1/many/{tokens}", (tokens, 2 * hkv, d), "bf16")
    kv = G.to_device(x, "bf16")
    table, lens = torch.arange(wide, dtype=torch.int32, device="cuda")[None], torch.tensor([tokens], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    binding.fa2_kv_append(p.k, p.v, kv[:, :hkv], kv[:, hkv:], table, lens, cu_new=cu, **p.kw())
    out = [torch.empty(1, hkv, tokens, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    binding.fa2_kv_read(p.k, p.v, *out, table, lens, **p.kw())
    binding.fa2_device_status()
    w = synth.widen(x, "bf16").transpose(1, 0, 2)
    for side, first, o in (("k", 0, out[0]), ("v", hkv, out[1])):
        for t in {0, tokens // 2, tokens - 1}:
            for h in range(hkv):
                assert np.array_equal(G.to_f64(o)[0, h, t], S.row_values4(*S.quantise_row4(w[first + h, t])))
        # scale within 2^-4 of a sixth of the largest; values past 6 scales, or half a step of 2 scales at most, off
        big = np.abs(w[first:first + hkv].reshape(hkv, tokens, -1, 16)).max(-1).repeat(16, -1)
        assert np.all(np.abs(G.to_f64(o)[0] - w[first:first + hkv]) <= big * (1 / 6 * (1 + 2.0 ** -4) + UNIT_ROUNDOFF["bf16"]))


def test_bad_pages_and_positions_are_not_stored():
    torch = G.require_gpu()
    p = Pools(3, 1, 16, 64)
    kv = G.to_device(synth.tensor("e2m1/bad", (4, 1, 64), "bf16"), "bf16")
    table = torch.tensor([[7, 0], [-1, 0], [1, 2], [1, 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([3, 16, 33, -2], dtype=torch.int32, device="cuda")
    binding.fa2_kv_append(p.k, p.v, kv, kv, table, lens, **p.kw())
    with pytest.raises(binding.Fa2Error) as err:
        binding.fa2_device_status()
    assert err.value.status == 8
    for side in "kv":
        codes, scales, bytes_ = p.host(side)
        assert np.all(bytes_ == p.fill) and np.all(scales == p.fill)
