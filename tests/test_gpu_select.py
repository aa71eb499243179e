"""Bounds of pages and the pages they select, exactly the float64 oracle's; and the attention over the selected pages, within
test_gpu_decode.py's tolerance."""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.paged import Cache
from tests.paged4 import Cache4
from tests.test_gpu_decode import check, workspace

pytestmark = pytest.mark.gpu


def cache_of(form, tag, lens, page, hkv, d, dtype="bf16", order="hnd", stale=True, **kw):
    if form == "e2m1":
        return Cache4(tag, lens, page, hkv, d, dtype, order, stale=stale, **kw)
    return Cache(tag, lens, page, hkv, d, dtype, form == "e4m3", order, stale="nan" if stale else None, **kw)


def k_only(c):
    return {k: v for k, v in c.exps().items() if k.startswith("k")}


def make_bounds(c, cu=None, tokens=None, lens=None):
    """Guarded bounds and exponents after fa2_kv_bounds; cu None and tokens None: all tokens of every sequence are new."""
    import torch
    dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    if tokens is None:
        cu = np.concatenate([[0], np.cumsum(np.maximum(c.lens, 0))])
        tokens = max(1, int(cu[-1]))
    bounds, exps = G.Guarded((c.pages, c.hkv, 2, c.d), torch.int8), G.Guarded((c.pages, c.hkv), torch.uint8)
    binding.fa2_kv_bounds(c.dev["k"], bounds.t, exps.t, c.table_dev, c.lens_dev, tokens, cu_new=None if cu is None else dev(cu), **k_only(c))
    return bounds, exps, cu


def check_bounds(c, bounds, exps, cu):
    bounds.assert_intact("bounds")
    exps.assert_intact("exponents")
    got, byte = bounds.t.cpu().numpy().astype(np.int64), exps.t.cpu().numpy()
    left = np.ones(c.pages, dtype=bool)
    for (b, j), live in S.touched_pages(c.lens, cu, c.page, c.wide * c.page).items():
        page = int(c.table[b, j])
        if not 0 <= page < c.pages:
            continue
        left[page] = False
        for h in range(c.hkv):
            codes, e = S.page_bounds(c.host["k"][page, h, :live])
            assert byte[page, h] == e and np.array_equal(got[page, h], codes), (b, j, h)
    fill = np.array([0xA5], dtype=np.uint8)
    assert np.all(byte[left] == fill) and np.all(got[left] == fill.view(np.int8))


@pytest.mark.parametrize("form,d", [("same", 8), ("same", 40), ("same", 64), ("same", 128), ("e4m3", 16), ("e4m3", 80), ("e4m3", 128), ("e2m1", 32),
                                    ("e2m1", 96), ("e2m1", 128)])
@pytest.mark.parametrize("page,order", [(1, "hnd"), (7, "nhd"), (16, "nhd"), (64, "hnd"), (200, "hnd")])
def test_bounds(page, order, form, d):
    G.require_gpu()
    lens = [37, 0, 150, 1, 64]
    c = cache_of(form, f"bounds/{page}", lens, page, 3, d, "f16" if d % 3 else "bf16", order)
    check_bounds(c, *make_bounds(c))
    # only the last tokens are new, some sequences have none, rows before and behind belong to nobody
    new = [3, 0, 17, 1, 0]
    cu = np.concatenate([[4], 4 + np.cumsum(new)])
    check_bounds(c, *make_bounds(c, cu, int(cu[-1]) + 9))
    check_bounds(c, *make_bounds(c, None, len(lens)))
    binding.fa2_device_status()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_bounds_of_special_keys(dtype):
    torch = G.require_gpu()
    c = Cache("bounds/special", [5, 16, 16, 16], 16, 2, 16, dtype, stale="inf")
    rows = synth.widen(synth.tensor("bounds/special/x", (c.pages, 2, 16, 16), dtype), dtype)
    t = c.table[:, 0]
    rows[t[0], :, 5:] = np.inf                      # behind the length
    rows[t[1], 0, 3, 4], rows[t[1], 1, :, 2], rows[t[1], 1, 7, 7] = np.nan, np.nan, np.inf
    rows[t[2], 0], rows[t[2], 1] = 0.0, -0.0
    rows[t[3], 0] *= 2.0 ** -20 if dtype == "f16" else 2.0 ** -100
    rows[t[3], 1] = np.arange(16) * 127.0 / 15
    x = synth.to_storage(rows, dtype)
    c.dev["k"].copy_(G.to_device(x, dtype))
    c.host["k"] = synth.widen(x, dtype)
    check_bounds(c, *make_bounds(c))
    binding.fa2_device_status()
    assert torch.isnan(c.dev["k"][t[1], 1, 0, 2])


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
@pytest.mark.parametrize("spread", [1, 13, 14, 15, 60])
def test_bounds_of_rows_of_different_powers(spread, form):
    """Rows whose powers of two lie up to so far apart in a page: the smallest codes of the smallest rows count, where a page has no others."""
    torch = G.require_gpu()
    c = cache_of(form, "bounds/powers", [200, 31], 16, 2, 64, stale=False)
    exps = c.exps()["k_exp"]
    up = (synth.counter_u16(f"bounds/powers/{spread}", tuple(exps.shape)) % (spread + 1)).astype(np.int64)
    up[:, :, 0], up[:, :, 1] = 0, spread  # the whole spread in each page
    exps += torch.from_numpy(up.astype(np.uint8)).cuda()
    c.host["k"] = c.host["k"] * 2.0 ** up[..., None]
    # a channel that is 0 but in the row of the lowest power, whose smallest code it has
    small = 2.0 ** (exps[:, :, 0].cpu().numpy().astype(np.float64) - 127)
    if form == "e4m3":
        codes = c.dev["k"].view(torch.uint8)
        codes[..., 5] = 0
        codes[:, :, 0, 5] = 1
        c.host["k"][..., 5], c.host["k"][:, :, 0, 5] = 0.0, 2.0 ** -9 * small
    check_bounds(c, *make_bounds(c))
    binding.fa2_device_status()


def test_bounds_skip_bad_pages_and_positions():
    torch = G.require_gpu()
    c = Cache("bounds/bad", [40, 40, 20], 16, 2, 32)
    c.table[0, 1], c.table[1, 0] = c.pages, -3
    c.table_dev.copy_(torch.from_numpy(c.table))
    got = make_bounds(c)
    with pytest.raises(binding.Fa2Error) as err:
        binding.fa2_device_status()
    assert err.value.status == 8
    check_bounds(c, *got)
    c = Cache("bounds/bad", [40, 40, 20], 16, 2, 32)
    c.lens = [1000, -4, 5]
    c.lens_dev.copy_(torch.tensor(c.lens, dtype=torch.int32))
    cu = [0, 970, 971, 981]
    got = make_bounds(c, cu, 981)
    with pytest.raises(binding.Fa2Error):
        binding.fa2_device_status()
    check_bounds(c, *got)


# ---------------------------------------------------------------------------- selection
def select(c, q, bounds, exps, budget, first, recent, fill=0xFF, stream=None):
    import torch
    batch, heads = q.shape[0], q.shape[1]
    table, lens = torch.full((batch, c.hkv, budget), -99, dtype=torch.int32, device="cuda"), torch.full((batch, c.hkv), -99, dtype=torch.int32, device="cuda")
    ws = G.Guarded((max(16, binding.fa2_select_workspace_size(batch, c.hkv, c.wide)),), torch.uint8)
    ws.t.fill_(fill)
    binding.fa2_select_pages(q, bounds, exps, c.table_dev, c.lens_dev, table, lens, ws.t, c.page, first=first, recent=recent, stream=stream)
    ws.assert_intact("workspace")
    return table, lens


def check_selection(c, q64, codes, byte, table, lens, budget, first, recent, rows=None):
    """Returns the numbers taken, {(sequence, head): [...]}."""
    got, got_lens = table.cpu().numpy(), lens.cpu().numpy()
    taken = {}
    group = q64.shape[1] // c.hkv
    for b in rows if rows is not None else range(len(c.lens)):
        n = min(max(c.lens[b], 0), c.wide * c.page)
        pages = c.table[b, : -(-n // c.page)]
        for h in range(c.hkv):
            scores = [S.page_score(q64[b, h * group:(h + 1) * group], codes[p, h], byte[p, h]) if 0 <= p < c.pages else None for p in pages]
            want = S.select_pages(scores, budget, first, recent)
            ids = [int(pages[j]) for j in want]
            assert got[b, h].tolist() == ids + [-1] * (budget - len(ids)), (b, h)
            held = len(want) * c.page - (len(pages) * c.page - n if want and want[-1] == len(pages) - 1 else 0)
            assert got_lens[b, h] == held
            taken[b, h] = want
    return taken


def run(form, tag, lens, page, hkv, group, d, budget, first=1, recent=1, dtype="bf16", order="hnd", rows=None, **kw):
    """Bounds, selection and attention of one call each; everything against the oracle."""
    torch = G.require_gpu()
    c = cache_of(form, tag, lens, page, hkv, d, dtype, order, **kw)
    bounds, exps, cu = make_bounds(c)
    heads = hkv * group
    full = synth.tensor(tag + "/q", (len(lens), heads + 2, d), dtype)
    q, q64 = G.to_device(full, dtype)[:, 1:heads + 1], synth.widen(full, dtype)[:, 1:heads + 1]
    table, sel_lens = select(c, q, bounds.t, exps.t, budget, first, recent)
    taken = check_selection(c, q64, bounds.t.cpu().numpy().astype(np.int64), exps.t.cpu().numpy(), table, sel_lens, budget, first, recent, rows)
    o, lse = G.guarded((len(lens), heads, d), dtype), G.guarded((len(lens), heads), "f32")
    scale = 1 / math.sqrt(d)
    binding.fa2_decode_selected(q, *c.pools(), o.t, lse.t, table, sel_lens, workspace(len(lens), heads, hkv, d), scale, **c.exps())
    binding.fa2_device_status()
    o.assert_intact("O")
    lse.assert_intact("LSE")
    for (b, h), want in taken.items():
        view = Selected(c, b, want)
        part = slice(h * group, (h + 1) * group)
        check(view.of_head(h), q64[b:b + 1, part], o.t[b:b + 1, part], lse.t[b:b + 1, part], group, scale)
    return c, q, table, sel_lens, o.t, lse.t


class Selected:
    """The selected pages of one sequence, of one key-value head, as check() takes a cache."""

    def __init__(self, c, b, want):
        self.c, self.b, self.want = c, b, want
        self.dtype, self.e4m3, self.d, self.lens = c.dtype, c.e4m3, c.d, [0]

    def of_head(self, h):
        self.h = h
        n = min(max(self.c.lens[self.b], 0), self.c.wide * self.c.page)
        self.at = [j * self.c.page + s for j in self.want for s in range(self.c.page) if j * self.c.page + s < n]
        return self

    def rows(self, side, b):
        rows, held = self.c.rows(side, self.b)
        return rows[self.at][:, self.h:self.h + 1], held[self.at]

    def value_exps(self, b, head):
        return self.c.value_exps(self.b, self.h)[self.at]


FORMS = ["same", "e4m3", "e2m1"]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("d", [128, 96, 64, 32])
def test_forms_and_head_sizes(d, form):
    run(form, f"sel/{d}", [300, 37, 1, 0, 160], 16, 2, 4, d, 5, dtype="bf16" if d % 64 else "f16", order="nhd" if d == 96 else "hnd")


@pytest.mark.parametrize("d", [8, 24, 40, 72, 120])
def test_head_sizes_of_half_chunks(d):
    run("same", f"sel/{d}", [300, 37], 16, 2, 2, d, 6, dtype="f16")


@pytest.mark.parametrize("page", [1, 5, 8, 24, 64, 100])
def test_page_sizes(page):
    run("same", f"sel/p{page}", [190, 64, 0, 7, 191], page, 2, 2, 64, max(2, 96 // page), order="nhd")
    run("e2m1", f"sel/p{page}", [190, 64, 0, 7, 191], page, 2, 2, 96, max(2, 96 // page))


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 9, 16, 20, 128])
def test_groups(group):
    run("same", f"sel/g{group}", [200, 33], 16, 2, group, 64, 4)


@pytest.mark.parametrize("budget,first,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (2, 1, 1), (3, 3, 0), (3, 0, 3), (7, 2, 3), (18, 0, 0), (19, 0, 0), (20, 1, 1), (500, 4, 4)])
def test_budgets(budget, first, recent):
    run("same", "sel/b", [300, 299, 16, 17, 0], 16, 2, 2, 32, budget, first, recent)


@pytest.mark.parametrize("n", [4000, 8100, 9001, 20000])
def test_many_pages(n):
    """More pages than a selecting CTA holds, and tables wider than the contexts."""
    run("same", f"sel/n{n}", [n, 5], 1, 1, 2, 32, 300, 1, 2, rows=[0, 1], stale=False, table_pages=n + (n % 3) * 1000)


def test_equal_scores_go_to_the_earliest():
    torch = G.require_gpu()
    c = Cache("sel/equal", [640, 100], 16, 2, 32)
    q = torch.ones(2, 4, 32, dtype=torch.bfloat16, device="cuda")
    bounds = torch.full((c.pages, 2, 2, 32), 3, dtype=torch.int8, device="cuda")
    exps = torch.full((c.pages, 2), 127, dtype=torch.uint8, device="cuda")
    for budget, first, recent in ((5, 0, 0), (5, 1, 2), (39, 0, 1)):
        table, lens = select(c, q, bounds, exps, budget, first, recent)
        check_selection(c, np.ones((2, 4, 32)), bounds.cpu().numpy().astype(np.int64), exps.cpu().numpy(), table, lens, budget, first, recent)
    binding.fa2_device_status()


def test_extreme_queries_and_bounds():
    """All codes' signs, powers of two far apart, scores past float32's range, zero queries, infinities and NaN in a query."""
    torch = G.require_gpu()
    c = Cache("sel/extreme", [1600] * 6, 16, 1, 64)
    raw = synth.counter_u16("sel/extreme/bounds", (c.pages, 1, 2, 64))
    codes = np.sort((raw % 255).astype(np.int64) - 127, axis=2)
    byte = (120 + synth.counter_u16("sel/extreme/exp", (c.pages, 1)) % 12).astype(np.uint8)
    byte[::7] = 67
    byte[::11] = 249
    q = synth.widen(synth.tensor("sel/extreme/q", (6, 3, 64), "bf16"), "bf16")
    q[1] *= 2.0 ** 100
    q[2] = 0
    q[3] *= 2.0 ** -100
    q[4, 0, :3] = np.inf, -np.inf, np.nan
    q[5] *= np.array([1.0, 2.0 ** -60, 2.0 ** 40])[:, None]
    x = synth.to_storage(q, "bf16")
    with np.errstate(over="ignore"):
        table, lens = select(c, G.to_device(x, "bf16"), torch.from_numpy(codes.astype(np.int8)).cuda(), torch.from_numpy(byte).cuda(), 20, 1, 1)
    binding.fa2_device_status()
    # float32 overflows to infinity: two such pages are alike
    exact = S.page_score

    def overflow(*a):
        s = exact(*a)
        return math.copysign(math.inf, s) if abs(s) >= 2.0 ** 128 else s
    S.page_score = overflow
    try:
        check_selection(c, synth.widen(x, "bf16"), codes, byte, table, lens, 20, 1, 1)
    finally:
        S.page_score = exact


def test_powers_that_are_none_select_within_the_budget():
    """Bytes 0 and 255 (bounds never made) stand for 0 and infinity: a score that is then no number is the lowest of a page of the
    cache, and no more pages than the budget are taken."""
    torch = G.require_gpu()
    c = Cache("sel/none", [1600, 1000, 1300], 16, 2, 64)
    codes = np.sort((synth.counter_u16("sel/none/bounds", (c.pages, 2, 2, 64)) % 255).astype(np.int64) - 127, axis=2)
    byte = np.array([0, 255, 127, 100], dtype=np.uint8)[synth.counter_u16("sel/none/exp", (c.pages, 2)) % 4]
    q = synth.widen(synth.tensor("sel/none/q", (3, 6, 64), "bf16"), "bf16")
    q[1], q[2] = 0, q[2] * 2.0 ** 120
    x = synth.to_storage(q, "bf16")

    def score(qs, codes, byte):
        best = max(S.page_score([one], codes, 127) for one in qs)
        best = math.copysign(math.inf, best) if abs(best) >= 2.0 ** 128 else best
        two = 0.0 if byte == 0 else math.inf if byte == 255 else 2.0 ** (int(byte) - 127)
        s = best * two
        return -math.inf if math.isnan(s) else s
    for budget, first, recent in ((20, 1, 1), (1, 0, 0), (60, 3, 9)):
        table, lens = select(c, G.to_device(x, "bf16"), torch.from_numpy(codes.astype(np.int8)).cuda(), torch.from_numpy(byte).cuda(), budget, first, recent)
        for b in range(3):
            pages = c.table[b, : -(-c.lens[b] // 16)]
            for h in range(2):
                scores = [score(synth.widen(x, "bf16")[b, 3 * h:3 * h + 3], codes[p, h], byte[p, h]) for p in pages]
                assert table[b, h].tolist() == [int(pages[j]) for j in S.select_pages(scores, budget, first, recent)], (b, h)
    binding.fa2_device_status()


@pytest.mark.parametrize("d", [128, 96, 40])
def test_the_largest_sums_are_exact(d):
    """Integers of 125 to 127 on both sides, all signs alike or nearly so: sums up to 2^21 that differ by little."""
    torch = G.require_gpu()
    c = Cache("sel/sums", [4000, 3999], 8, 2, d)
    raw = synth.counter_u16(f"sel/sums/{d}", (c.pages, 2, 2, d)).astype(np.int64)
    codes = np.where(np.arange(2)[:, None] == 1, 127 - raw % 3, 125 - raw % 3)
    codes[::2] = -codes[::2, :, ::-1]
    byte = np.full((c.pages, 2), 127, dtype=np.uint8)
    ints = 127.0 - synth.counter_u16(f"sel/sums/q{d}", (2, 6, d)) % 3
    ints[:, :, 0] = 127.0
    ints[0, ::2] *= -1
    ints[1, 1, ::7] *= -1
    x = synth.to_storage(ints, "bf16")
    for budget in (5, 100, 499):
        table, lens = select(c, G.to_device(x, "bf16"), torch.from_numpy(codes.astype(np.int8)).cuda(), torch.from_numpy(byte).cuda(), budget, 0, 1)
        check_selection(c, synth.widen(x, "bf16"), codes, byte, table, lens, budget, 0, 1)
    binding.fa2_device_status()


def test_bad_pages_come_last():
    torch = G.require_gpu()
    c = Cache("sel/bad", [320, 64], 16, 2, 32)
    bounds, exps, _ = make_bounds(c)
    c.table[0, 3], c.table[0, 19], c.table[1, 0] = -1, c.pages, 2 ** 31 - 1
    c.table_dev.copy_(torch.from_numpy(c.table))
    full = synth.tensor("sel/bad/q", (2, 4, 32), "bf16")
    for budget, first, recent in ((6, 0, 0), (19, 0, 0), (4, 1, 1), (100, 0, 0)):
        table, lens = select(c, G.to_device(full, "bf16"), bounds.t, exps.t, budget, first, recent)
        with pytest.raises(binding.Fa2Error) as err:
            binding.fa2_device_status()
        assert err.value.status == 8
        check_selection(c, synth.widen(full, "bf16"), bounds.t.cpu().numpy().astype(np.int64), exps.t.cpu().numpy(), table, lens, budget, first, recent)


def test_lengths_outside_the_table():
    torch = G.require_gpu()
    c = Cache("sel/lens", [64, 64, 64], 16, 1, 32)
    bounds, exps, _ = make_bounds(c)
    c.lens = [-3, 10 ** 6, 64]
    c.lens_dev.copy_(torch.tensor(c.lens, dtype=torch.int32))
    full = synth.tensor("sel/lens/q", (3, 2, 32), "bf16")
    table, lens = select(c, G.to_device(full, "bf16"), bounds.t, exps.t, 2, 0, 1)
    with pytest.raises(binding.Fa2Error):
        binding.fa2_device_status()
    check_selection(c, synth.widen(full, "bf16"), bounds.t.cpu().numpy().astype(np.int64), exps.t.cpu().numpy(), table, lens, 2, 0, 1)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("batch,hkv,group,budget", [(1, 8, 4, 128), (40, 8, 2, 4), (3, 4, 16, 200), (2, 1, 20, 40)])
def test_short_and_long_selections(batch, hkv, group, budget, form):
    """Selections that one launch of clusters takes and such that two launches divide."""
    lens = [(997 * i * i + 211 * i) % 2500 + 500 for i in range(batch)]
    run(form, "sel/short", lens, 16, hkv, group, 64, budget, 1, 2, rows=range(0, batch, 9), stale=False)


def test_same_bits_on_another_stream_and_with_other_workspaces():
    torch = G.require_gpu()
    c, q, table, lens, o, lse = run("e2m1", "sel/again", [3000, 77, 900], 16, 2, 4, 128, 20)
    bounds, exps, _ = make_bounds(c)
    side = torch.cuda.Stream()
    for fill in (0, 0x7F):
        torch.cuda.synchronize()
        t2, l2 = select(c, q, bounds.t, exps.t, 20, 1, 1, fill, side)
        ws, o2, lse2 = workspace(3, 8, 2, 128, fill), torch.full_like(o, 5.0), torch.full_like(lse, 5.0)
        torch.cuda.synchronize()
        binding.fa2_decode_selected(q, *c.pools(), o2, lse2, t2, l2, ws, 1 / math.sqrt(128), stream=side, **c.exps())
        side.synchronize()
        assert torch.equal(table, t2) and torch.equal(lens, l2) and torch.equal(o, o2) and torch.equal(lse, lse2)
