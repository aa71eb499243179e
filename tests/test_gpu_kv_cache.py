"""Writing to and reading from the paged cache on the GPU: bit for bit what the oracle says.

16-bit rows are copied; an e4m3 code is the nearest one to x / 2^e, a quotient without rounding, so code and scale byte
are determined, and code * 2^e is exact in bfloat16 and, for the sizes here, in half.
"""
import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.paged import Cache

pytestmark = pytest.mark.gpu


def rows_for(tag, total, hkv, d, dtype):
    """Rows with a spread of sizes, zero rows, and infinities and NaN among the last ones."""
    x = synth.normal(3, tag, total * hkv * d).reshape(total, hkv, d)
    x = x * 2.0 ** (np.arange(total) % 9 - 4)[:, None, None]
    x[0, 0] = 0
    x[total // 2, :, : d // 2] = 448.0
    if total > 2:
        x[-1, 0, 1], x[-1, -1, 2], x[-1, -1, 3] = np.inf, -np.inf, np.nan
    return synth.to_storage(x, dtype)


def bits(t):
    import torch
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu().numpy()


CASES = [
    # lens, new, page, hkv, d, dtype, e4m3, order
    ([5], None, 16, 1, 128, "bf16", False, "hnd"),
    ([1, 17, 33, 16], None, 16, 8, 128, "bf16", True, "hnd"),
    ([40, 7, 1, 65], [40, 3, 1, 2], 16, 3, 64, "f16", True, "nhd"),
    ([40, 7, 1, 65], [13, 0, 1, 65], 24, 2, 80, "bf16", True, "hnd"),
    ([300, 129], [300, 128], 64, 5, 96, "f16", False, "nhd"),
    ([9, 4], [9, 4], 1, 4, 32, "bf16", True, "hnd"),
    ([9, 4, 12], [9, 1, 5], 5, 1, 8, "f16", False, "hnd"),
    ([9, 4, 12], [9, 1, 5], 1000, 2, 16, "f16", True, "nhd"),
    ([700, 1500, 33], [700, 900, 33], 32, 16, 112, "bf16", True, "nhd"),
    ([6], [6], 8, 70, 24, "bf16", False, "nhd"),
    ([2000, 3001], [2000, 3000], 128, 2, 128, "bf16", False, "hnd"),
    # few heads: several tokens a warp at once, with few and with many tokens
    ([40, 7, 1, 65], [40, 3, 1, 2], 16, 1, 64, "bf16", True, "hnd"),
    ([9000, 1, 4100], [9000, 1, 4099], 16, 1, 32, "bf16", True, "hnd"),
    ([20000], [19999], 64, 3, 16, "f16", False, "nhd"),
    ([6000, 2], [6000, 2], 24, 2, 48, "f16", True, "nhd"),
    ([5000], [5000], 16, 1, 112, "f16", True, "nhd"),
]


@pytest.mark.parametrize("lens,new,page,hkv,d,dtype,e4m3,order", CASES)
def test_append(lens, new, page, hkv, d, dtype, e4m3, order):
    torch = G.require_gpu()
    tag = f"append/{lens}/{page}/{d}"
    c = Cache(tag, lens, page, hkv, d, dtype, e4m3, order)
    cu = None if new is None else np.concatenate([[0], np.cumsum(new)])
    total = len(lens) if new is None else int(cu[-1])
    behind = 0 if new is None else 3  # rows past the last sequence: not stored
    kv = [rows_for(tag + s, total + behind, hkv, d, dtype) for s in "kv"]
    both = torch.cat([G.to_device(x, dtype) for x in kv], 1)  # slices of one projection
    want = {s: bits(c.dev[s]).copy() for s in "kv"}
    want_exp = {s: c.exp[s].cpu().numpy().copy() for s in "kv"} if e4m3 else {}
    for s, x in zip("kv", kv):
        wide = synth.widen(x, dtype)
        raw = x if dtype == "bf16" else x.view(np.uint16)
        for t, p, slot in S.append_slots(c.table, lens, cu, page, c.pages):
            for h in range(hkv):
                if e4m3:
                    want[s][p, h, slot], want_exp[s][p, h, slot] = S.quantise_row(wide[t, h])
                else:
                    want[s][p, h, slot] = raw[t, h].view(np.int16)
    cu_dev = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    binding.fa2_kv_append(*c.pools(), both[:, :hkv], both[:, hkv:], c.table_dev, c.lens_dev, cu_new=cu_dev, **c.exps())
    binding.fa2_device_status()
    for s in "kv":
        got = bits(c.dev[s])
        if e4m3:  # the sign of a NaN says nothing
            got, ref = (np.where((a & 127) == 127, 127, a) for a in (got, want[s]))
            assert np.array_equal(c.exp[s].cpu().numpy(), want_exp[s])
        else:
            ref = want[s]
        assert np.array_equal(got, ref), f"{s}: {np.argwhere(got != ref)[:5]}"


@pytest.mark.parametrize("lens,page,hkv,d,dtype,e4m3,order,out", [
    ([5], 16, 1, 128, "bf16", False, "hnd", "bhnd"), ([1, 0, 33, 16], 16, 8, 128, "bf16", True, "hnd", "bhnd"),
    ([40, 7, 1, 65], 24, 3, 64, "f16", True, "nhd", "bnhd"), ([300, 129], 64, 5, 96, "f16", False, "nhd", "bnhd"),
    ([9, 4, 12], 1, 2, 16, "f16", True, "nhd", "bhnd"), ([9, 4, 12], 1000, 4, 8, "bf16", False, "hnd", "bnhd"),
    ([700, 1500, 33], 32, 16, 112, "bf16", True, "nhd", "bhnd"), ([2000, 3001], 128, 2, 128, "bf16", True, "hnd", "bhnd"),
    ([20000, 0, 777], 16, 1, 32, "bf16", True, "hnd", "bhnd"), ([9000, 9100], 64, 3, 16, "f16", False, "nhd", "bnhd"),
    ([50], 8, 2, 40, "bf16", False, "hnd", "bnhd"),
])
@pytest.mark.parametrize("cut", [False, True])
def test_read(lens, page, hkv, d, dtype, e4m3, order, out, cut):
    torch = G.require_gpu()
    c = Cache(f"read/{lens}/{page}", lens, page, hkv, d, dtype, e4m3, order, stale="nan")
    n = max(1, max(lens) - 2) if cut else max(lens) + 3
    shape = (len(lens), hkv, n, d) if out == "bhnd" else (len(lens), n, hkv, d)
    outs = [G.guarded(shape, dtype) for _ in "kv"]
    views = [g.t if out == "bhnd" else g.t.transpose(1, 2) for g in outs]
    binding.fa2_kv_read(*c.pools(), *views, c.table_dev, c.lens_dev, **c.exps())
    binding.fa2_device_status()
    for s, g, t in zip("kv", outs, views):
        g.assert_intact(s)
        got = G.to_f64(t)
        for b, length in enumerate(lens):
            m = min(length, n)
            rows, _ = c.rows(s, b)
            assert np.array_equal(got[b, :, :m], rows[:m].swapaxes(0, 1))
            assert np.all(np.isnan(got[b, :, m:]))  # left as they were: the guard's pattern


def test_round_trip_error():
    """A row read back is within half an e4m3 step (2^-4 of the value, or of the row's smallest step) of what was written."""
    torch = G.require_gpu()
    c = Cache("trip", [50], 16, 4, 64, "bf16", True)
    x = synth.tensor("trip/x", (50, 4, 64), "bf16")
    xd = G.to_device(x, "bf16")
    cu = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    binding.fa2_kv_append(*c.pools(), xd, xd, c.table_dev, c.lens_dev, cu_new=cu, **c.exps())
    k, v = G.empty((1, 4, 50, 64), "bf16"), G.empty((1, 4, 50, 64), "bf16")
    binding.fa2_kv_read(*c.pools(), k, v, c.table_dev, c.lens_dev, **c.exps())
    w = synth.widen(x, "bf16").swapaxes(0, 1)[None]
    step = np.max(np.abs(w), -1, keepdims=True) / 224 * 2.0 ** -10  # scale <= max / 224; half of its smallest step 2^-9
    assert np.all(np.abs(G.to_f64(k) - w) <= np.maximum(2.0 ** -4 * np.abs(w), step)) and torch.equal(k, v)


@pytest.mark.parametrize("e4m3", [False, True])
def test_bad_pages_and_lengths(e4m3):
    """Page numbers outside the pool, lengths outside the table, new tokens before a sequence's start: nothing of theirs is
    written or read, the rest is, and the status says so once."""
    torch = G.require_gpu()
    lens = [40, 35, 20]
    c = Cache("bad", lens, 16, 2, 32, "bf16", e4m3)
    c.table[0, 1], c.table[1, 0], c.table[2, 1] = c.pages, -1, 2 ** 31 - 1
    c.table_dev.copy_(torch.from_numpy(c.table))
    k, v = (G.empty((3, 2, 40, 32), "bf16").fill_(5.0) for _ in "kv")
    binding.fa2_kv_read(*c.pools(), k, v, c.table_dev, c.lens_dev, **c.exps())
    with pytest.raises(binding.Fa2Error) as err:
        binding.fa2_device_status()
    assert err.value.status == 8
    binding.fa2_device_status()  # cleared
    for b in range(3):
        rows, held = c.rows("k", b)
        got = G.to_f64(k)[b].swapaxes(0, 1)
        assert np.array_equal(got[: lens[b]][held], rows[held]) and np.all(got[: lens[b]][~held] == 5.0) and np.all(got[lens[b]:] == 5.0)
    # append: sequence 0 has 4 new tokens but a length of 2, sequence 1 passes its table, sequence 2 has a negative length
    new_lens, cu = [2, 50, -3], [0, 4, 7, 9]
    x = synth.tensor("bad/new", (9, 2, 32), "bf16")
    xd = G.to_device(x, "bf16")
    before = bits(c.dev["k"]).copy()
    binding.fa2_kv_append(*c.pools(), xd, xd, c.table_dev, torch.tensor(new_lens, dtype=torch.int32, device="cuda"),
                          cu_new=torch.tensor(cu, dtype=torch.int32, device="cuda"), **c.exps())
    with pytest.raises(binding.Fa2Error):
        binding.fa2_device_status()
    slots = S.append_slots(c.table, new_lens, cu, 16, c.pages)
    assert [s[0] for s in slots] == [2, 3, 4]  # tokens 0, 1 have no position; 4 has one (47); 5, 6 pass the table; 7, 8 have none
    touched = np.zeros(before.shape[:3], bool)
    for _, p, s in slots:
        touched[p, :, s] = True
    assert np.array_equal(bits(c.dev["k"])[~touched], before[~touched])
    k2, v2 = (G.empty((3, 2, 48, 32), "bf16") for _ in "kv")
    binding.fa2_kv_read(*c.pools(), k2, v2, c.table_dev, torch.tensor([2, 99, -1], dtype=torch.int32, device="cuda"), **c.exps())
    with pytest.raises(binding.Fa2Error):
        binding.fa2_device_status()
    ref = synth.widen(x, "bf16")
    if e4m3:
        ref = np.array([[S.row_values(*S.quantise_row(r)) for r in t] for t in ref])
    assert np.array_equal(G.to_f64(k2)[0, :, :2].swapaxes(0, 1), ref[2:4])
    assert np.array_equal(G.to_f64(k2)[1, :, 47], ref[4])


def test_a_sequence_of_length_zero_stores_nothing():
    torch = G.require_gpu()
    c = Cache("zero", [3, 0, 2], 4, 2, 32, "bf16", True)
    before = bits(c.dev["v"]).copy()
    xd = G.to_device(synth.tensor("zero/x", (3, 2, 32), "bf16"), "bf16")
    binding.fa2_kv_append(*c.pools(), xd, xd, c.table_dev, c.lens_dev, **c.exps())
    binding.fa2_device_status()
    changed = np.argwhere((bits(c.dev["v"]) != before).any((1, 3)))
    assert {tuple(x) for x in changed} == {(c.table[0, 0], 2), (c.table[2, 0], 1)}


@pytest.mark.parametrize("e4m3", [False, True])
def test_offsets_past_2_32_bytes(e4m3):
    """Pages on both sides of 4 GiB of a pool, through wide page strides."""
    torch = G.require_gpu()
    hkv, page, d, size = 2, 16, 64, 1 if e4m3 else 2
    stride = ((1 << 32) + 4096) // size // 2
    bufs = [torch.zeros(2 * stride + hkv * page * d, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda") for _ in "kv"]
    pools = [b.as_strided((3, hkv, page, d), (stride, page * d, d, 1)) for b in bufs]
    pools = [p.view(torch.float8_e4m3fn) if e4m3 else p for p in pools]
    exps = {f"{s}_exp": torch.zeros(3, hkv, page, dtype=torch.uint8, device="cuda") for s in "kv"} if e4m3 else {}
    table, lens = torch.tensor([[2, 0], [1, 0]], dtype=torch.int32, device="cuda"), torch.tensor([20, 16], dtype=torch.int32, device="cuda")
    x = synth.tensor("far/x", (36, hkv, d), "bf16")
    xd = G.to_device(x, "bf16")
    cu = torch.tensor([0, 20, 36], dtype=torch.int32, device="cuda")
    binding.fa2_kv_append(*pools, xd, -xd, table, lens, cu_new=cu, **exps)
    k, v = G.empty((2, hkv, 20, d), "bf16"), G.empty((2, hkv, 20, d), "bf16")
    binding.fa2_kv_read(*pools, k, v, table, lens, **exps)
    binding.fa2_device_status()
    ref = synth.widen(x, "bf16")
    if e4m3:
        ref = np.array([[S.row_values(*S.quantise_row(r)) for r in t] for t in ref])
    for b, (at, n) in enumerate(((0, 20), (20, 16))):
        assert np.array_equal(G.to_f64(k)[b, :, :n].swapaxes(0, 1), ref[at:at + n])
        assert np.array_equal(G.to_f64(v)[b, :, :n].swapaxes(0, 1), -ref[at:at + n])
