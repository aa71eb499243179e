"""The rotated append, the bounds, the selection and its attention run together, as a program that generates tokens uses them."""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.test_gpu_decode import check
from tests.test_gpu_rope_append import Pages
from tests.test_gpu_select import Selected

pytestmark = pytest.mark.gpu

HKV, GROUP, D, PAGE, BUDGET = 2, 3, 64, 16, 4
HEADS = HKV * GROUP
FORMS = ["same", "e4m3", "e2m1"]


class Server:
    """Prompts of given lengths, then tokens one by one: the projections are seeded, everything after them the library's."""

    def __init__(self, form, prompts, steps, budget=BUDGET):
        torch = G.require_gpu()
        self.form, self.prompts, self.steps = form, prompts, steps
        batch, wide = len(prompts), -(-(max(prompts) + steps) // PAGE)
        self.pages = Pages(form, batch * wide + 1, HKV, PAGE, D, "bf16")
        self.table = torch.from_numpy(np.argsort(synth.raw_words(5, "sparse/server", 0, batch * wide + 1), kind="stable")[: batch * wide]
                                      .reshape(batch, wide).astype(np.int32)).cuda()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        freq, self.magnitude = binding.fa2_rope_frequencies(D, 10000.0, "ramp", 4.0, 32.0)
        self.freq64, self.freq = freq.numpy(), freq.cuda()
        self.qkv = [synth.tensor(f"sparse/server/{b}", (n + steps, HEADS + 2 * HKV, D), "bf16") for b, n in enumerate(prompts)]
        self.bounds = torch.zeros(self.pages.pages, HKV, 2, D, dtype=torch.int8, device="cuda")
        self.bounds_exp = torch.zeros(self.pages.pages, HKV, dtype=torch.uint8, device="cuda")
        self.sel = torch.empty(batch, HKV, budget, dtype=torch.int32, device="cuda")
        self.sel_lens = torch.empty(batch, HKV, dtype=torch.int32, device="cuda")
        self.ws_select = torch.empty(binding.fa2_select_workspace_size(batch, HKV, wide), dtype=torch.uint8, device="cuda")
        self.ws = torch.empty(binding.fa2_decode_workspace_size(batch, HEADS, HKV, D), dtype=torch.uint8, device="cuda")
        self.o, self.lse = G.empty((batch, HEADS, D), "bf16"), torch.empty(batch, HEADS, device="cuda")

    def store(self, rows, cu=None):
        """rows [T, HEADS + 2 HKV, D]: q turned in place, k and v stored, the bounds of their pages made."""
        q, k, v = rows[:, :HEADS], rows[:, HEADS:HEADS + HKV], rows[:, HEADS + HKV:]
        kw = self.pages.kw
        binding.fa2_rope_append(*self.pages.pools, k, v, self.freq, self.table, self.lens, q=q, q_out=q, cu_new=cu, magnitude=self.magnitude, **kw)
        binding.fa2_kv_bounds(self.pages.pools[0], self.bounds, self.bounds_exp, self.table, self.lens, rows.shape[0], cu_new=cu,
                              k_exp=kw.get("k_exp"), k_scale=kw.get("k_scale"))

    def prefill(self):
        torch = G.require_gpu()
        rows = torch.cat([G.to_device(x[:n], "bf16") for x, n in zip(self.qkv, self.prompts)])
        self.lens.copy_(torch.tensor(self.prompts, dtype=torch.int32))
        self.store(rows, torch.tensor(np.concatenate([[0], np.cumsum(self.prompts)]), dtype=torch.int32, device="cuda"))

    def step(self, rows):
        self.store(rows)
        q = rows[:, :HEADS]
        binding.fa2_select_pages(q, self.bounds, self.bounds_exp, self.table, self.lens, self.sel, self.sel_lens, self.ws_select, PAGE)
        binding.fa2_decode_selected(q, *self.pages.pools, self.o, self.lse, self.sel, self.sel_lens, self.ws, 1 / math.sqrt(D), **self.pages.kw)

    def new_rows(self, i):
        return np.stack([x[n + i] for x, n in zip(self.qkv, self.prompts)])


class Held:
    """A server's cache as the selection's check takes one: its rows as they are stored."""

    def __init__(self, s):
        self.s, self.page, self.hkv, self.d, self.dtype, self.e4m3 = s, PAGE, HKV, D, "bf16", s.form != "same"
        self.pages, self.table, self.lens = s.pages.pages, s.table.cpu().numpy(), s.lens.cpu().tolist()
        self.wide = self.table.shape[1]

    def rows(self, side, b):
        at = [(int(self.table[b, p // PAGE]), p % PAGE) for p in range(self.lens[b])]
        return np.array([[self.s.pages.row(side, (pg, h, slot))[0] for h in range(HKV)] for pg, slot in at]), np.ones(len(at), dtype=bool)

    def value_exps(self, b, h):
        if self.s.form == "same":
            return np.zeros(self.lens[b])
        return np.array([int(self.s.pages.kw["v_exp"][int(self.table[b, p // PAGE]), h, p % PAGE]) - 127 for p in range(self.lens[b])])


@pytest.mark.parametrize("form", FORMS)
def test_generation_reads_the_pages_its_bounds_select(form):
    """After every step: the bounds are those of the keys in the cache, the pages taken those the bounds select, and the
    attention that over their rows."""
    s = Server(form, [100, 1, 64, 33], 18)
    s.prefill()
    for i in range(s.steps):
        s.lens += 1
        rows = G.to_device(s.new_rows(i), "bf16")
        s.step(rows)
        binding.fa2_device_status()
        if i % 6:
            continue
        c, q = Held(s), G.to_f64(rows[:, :HEADS])
        codes, byte = s.bounds.cpu().numpy().astype(np.int64), s.bounds_exp.cpu().numpy()
        for b, n in enumerate(c.lens):
            k = c.rows("k", b)[0]
            for h in range(HKV):
                ids = c.table[b, : -(-n // PAGE)]
                for j, page in enumerate(ids):
                    want = S.page_bounds(k[j * PAGE:(j + 1) * PAGE, h])
                    assert np.array_equal(codes[page, h], want[0]) and byte[page, h] == want[1]
                part = slice(h * GROUP, (h + 1) * GROUP)
                taken = S.select_pages([S.page_score(q[b, part], codes[p, h], byte[p, h]) for p in ids], BUDGET, 1, 1)
                got = s.sel[b, h].cpu().tolist()
                assert got == [int(ids[j]) for j in taken] + [-1] * (BUDGET - len(taken))
                check(Selected(c, b, taken).of_head(h), q[b:b + 1, part], s.o[b:b + 1, part], s.lse[b:b + 1, part], GROUP, 1 / math.sqrt(D))


@pytest.mark.parametrize("form", FORMS)
def test_with_room_for_every_page_it_is_the_whole_attention(form):
    """A budget of all pages: fa2_decode's result, but for the division of the work (tolerances as there, twice)."""
    torch = G.require_gpu()
    s = Server(form, [300, 7], 1, budget=32)
    s.prefill()
    s.lens += 1
    rows = G.to_device(s.new_rows(0), "bf16")
    s.step(rows)
    o, lse = torch.empty_like(s.o), torch.empty_like(s.lse)
    binding.fa2_decode(rows[:, :HEADS], *s.pages.pools, o, lse, s.table, s.lens, s.ws, 1 / math.sqrt(D), **s.pages.kw)
    binding.fa2_device_status()
    c, q = Held(s), G.to_f64(rows[:, :HEADS])
    for got in ((s.o, s.lse), (o, lse)):
        for b in range(2):
            for h in range(HKV):
                part = slice(h * GROUP, (h + 1) * GROUP)
                check(Selected(c, b, range(-(-c.lens[b] // PAGE))).of_head(h), q[b:b + 1, part], got[0][b:b + 1, part], got[1][b:b + 1, part], GROUP,
                      1 / math.sqrt(D))


@pytest.mark.parametrize("form", FORMS)
def test_a_captured_step_replays_with_new_lengths(form):
    """One graph of a whole step replayed for every token gives what the eager calls give, bit for bit."""
    torch = G.require_gpu()
    a, b = (Server(form, [100, 1, 64, 33], 12) for _ in range(2))
    a.prefill()
    b.prefill()
    rows = torch.empty(4, HEADS + 2 * HKV, D, dtype=torch.bfloat16, device="cuda")

    def one():
        b.lens += 1
        b.step(rows)

    rows.copy_(G.to_device(b.new_rows(0), "bf16"))
    before = b.lens.clone()
    one()  # eager once, for the library's one-time settings
    torch.cuda.synchronize()
    b.lens.copy_(before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    for i in range(a.steps):
        a.lens += 1
        a.step(G.to_device(a.new_rows(i), "bf16"))
        rows.copy_(G.to_device(b.new_rows(i), "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.sel, b.sel) and torch.equal(a.sel_lens, b.sel_lens) and torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse), i
    assert torch.equal(a.bounds, b.bounds) and torch.equal(a.pages.raw[0], b.pages.raw[0]) and torch.equal(a.pages.raw[1], b.pages.raw[1])
    binding.fa2_device_status()
