"""Calls of the rotated append, the bounds and the selection that their documentation allows and the other tests do not make."""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import serving as S
from tests import gpu_util as G
from tests.paged import Cache
from tests.test_gpu_rope_append import Pages
from tests.test_gpu_select import check_bounds, check_selection, make_bounds, select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["same", "e4m3", "e2m1"])
def test_the_append_alone_and_the_rotated_one_store_the_same_values(form):
    """Values do not turn: both calls store the same bits for them, and a rotation by nothing (position 0) stores the same keys in 16
    bits, and in 4 bits with a magnitude of 1."""
    torch = G.require_gpu()
    a, b = (Pages(form, 3, 2, 16, 64, "bf16") for _ in range(2))
    rows = G.to_device(synth.tensor("paths/same", (40, 4, 64), "bf16"), "bf16")
    table, lens = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda"), torch.tensor([40], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    freq, _ = binding.fa2_rope_frequencies(64)
    binding.fa2_kv_append(*a.pools, rows[:, :2], rows[:, 2:], table, lens, cu_new=cu, **a.kw)
    binding.fa2_rope_append(*b.pools, rows[:, :2], rows[:, 2:], freq.cuda(), table, lens, cu_new=cu,
                            positions=torch.zeros(40, dtype=torch.int32, device="cuda"), **b.kw)
    binding.fa2_device_status()
    assert torch.equal(a.raw[1], b.raw[1])
    if form != "same":
        assert torch.equal(a.kw["v_exp"], b.kw["v_exp"])
    if form != "e4m3":
        assert torch.equal(a.raw[0] & 0x77 if form == "e2m1" else a.raw[0], b.raw[0] & 0x77 if form == "e2m1" else b.raw[0])


@pytest.mark.parametrize("form", ["same", "e4m3", "e2m1"])
def test_strided_rows_and_streams(form):
    """Rows with strides of their own for q, q_out, k and v, a stride of 0 among them, on a side stream."""
    torch = G.require_gpu()
    t, h, hkv, d = 9, 3, 2, 64
    base = G.to_device(synth.tensor("paths/strided", (t, 8, 2 * d), "bf16"), "bf16")
    q, k = base[:, 2:5, d:], base[:1, :2, :d].expand(t, hkv, d)  # every token the same key row
    v = base[:, 6:8, :d]
    out = torch.full((h, t, 2 * d), float("nan"), dtype=torch.bfloat16, device="cuda")
    q_out = out[:, :, :d].transpose(0, 1)
    freq, _ = binding.fa2_rope_frequencies(d)
    table, lens = torch.tensor([[0]], dtype=torch.int32, device="cuda"), torch.tensor([t], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, t], dtype=torch.int32, device="cuda")
    freq = freq.cuda()
    one, two = Pages(form, 1, hkv, 16, d, "bf16"), Pages(form, 1, hkv, 16, d, "bf16")
    dense = torch.empty(t, h, d, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    binding.fa2_rope_append(*one.pools, k, v, freq, table, lens, q=q, q_out=q_out, cu_new=cu, stream=side, **one.kw)
    side.synchronize()
    binding.fa2_rope_append(*two.pools, k.contiguous(), v.contiguous(), freq, table, lens, q=q.contiguous(), q_out=dense, cu_new=cu, **two.kw)
    binding.fa2_device_status()
    assert torch.equal(q_out, dense) and torch.isnan(out[:, :, d:]).all()
    assert torch.equal(one.raw[0], two.raw[0]) and torch.equal(one.raw[1], two.raw[1])


def test_rows_of_a_call_that_one_sequence_fills_alone():
    """Sequences without new tokens at both ends and between; one whose new tokens end in the middle of a page."""
    torch = G.require_gpu()
    c = Cache("paths/ends", [20, 0, 35, 7], 16, 2, 32)
    new = [0, 0, 35, 0]
    check_bounds(c, *make_bounds(c, np.concatenate([[0], np.cumsum(new)]), 35))
    binding.fa2_device_status()
    assert torch.equal(c.lens_dev.cpu(), torch.tensor([20, 0, 35, 7], dtype=torch.int32))


@pytest.mark.parametrize("wide", [12287, 12288, 12300, 40000])
def test_tables_that_one_launch_takes_and_that_two_take(wide):
    """One sequence of up to so many pages of one token, and of few."""
    torch = G.require_gpu()
    for n in (wide - 1, 700):
        c = Cache("paths/wide", [n], 1, 1, 8, stale=None, table_pages=wide)
        raw = synth.counter_u16(f"paths/wide/{wide}", (c.pages, 1, 2, 8)).astype(np.int64)
        codes, byte = np.sort(raw % 255 - 127, axis=2), np.full((c.pages, 1), 127, dtype=np.uint8)
        full = synth.tensor("paths/wide/q", (1, 2, 8), "bf16")
        table, lens = select(c, G.to_device(full, "bf16"), torch.from_numpy(codes.astype(np.int8)).cuda(), torch.from_numpy(byte).cuda(), 600, 2, 3)
        binding.fa2_device_status()
        got = table.cpu().numpy()[0, 0]
        # scores of all pages at once (the oracle's page by page is slow here)
        ints, e = zip(*(S.query_integers(x) for x in synth.widen(full, "bf16")[0]))
        ids = c.table[0, :n]
        u = np.stack([np.maximum(i * codes[ids, 0, 0], i * codes[ids, 0, 1]).sum(1) * 2.0 ** x for i, x in zip(ints, e)]).max(0)
        assert got.tolist() == [int(ids[j]) for j in S.select_pages(list(u), 600, 2, 3)] and lens.item() == 600


@pytest.mark.parametrize("groups", [1, 7, 128])
def test_the_largest_groups_and_rows(groups):
    """As many query heads as a call takes, at the largest head size; rows of more sequences and heads than CTAs."""
    G.require_gpu()
    c = Cache("paths/groups", [130] * (3 if groups == 128 else 60), 8, 4, 128, "f16", stale=None)
    bounds, exps, _ = make_bounds(c)
    full = synth.tensor("paths/groups/q", (len(c.lens), 4 * groups, 128), "f16")
    table, lens = select(c, G.to_device(full, "f16"), bounds.t, exps.t, 5, 1, 1)
    binding.fa2_device_status()
    check_selection(c, synth.widen(full, "f16"), bounds.t.cpu().numpy().astype(np.int64), exps.t.cpu().numpy(), table, lens, 5, 1, 1,
                    rows=[0, len(c.lens) - 1])


def test_two_steps_at_once_on_two_streams():
    """Two independent steps (stores, bounds, selection, attention) whose kernels overlap give what they give alone."""
    torch = G.require_gpu()
    from tests.test_gpu_sparse_serving import Server
    alone = [Server(f, [300, 41, 7], 3) for f in ("e2m1", "same")]
    for s in alone:
        s.prefill()
    rows = [[G.to_device(s.new_rows(i), "bf16") for i in range(3)] for s in alone]
    for s, r in zip(alone, rows):
        for x in r:
            s.lens += 1
            s.step(x.clone())
    both = [Server(f, [300, 41, 7], 3) for f in ("e2m1", "same")]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for s, stream in zip(both, streams):
        with torch.cuda.stream(stream):
            s.prefill()
    for i in range(3):
        for s, r, stream in zip(both, rows, streams):
            with torch.cuda.stream(stream):
                s.lens += 1
                s.step(r[i].clone())
    torch.cuda.synchronize()
    binding.fa2_device_status()
    for a, b in zip(alone, both):
        assert torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse) and torch.equal(a.sel, b.sel) and torch.equal(a.bounds, b.bounds)


def test_a_step_captured_without_an_eager_one():
    """The first call of a size may be the captured one."""
    torch = G.require_gpu()
    c = Cache("paths/capture", [1000, 77], 16, 5, 72, "f16")
    bounds, exps, _ = make_bounds(c)
    q = G.to_device(synth.tensor("paths/capture/q", (2, 15, 72), "f16"), "f16")
    sel, sel_lens = torch.empty(2, 5, 9, dtype=torch.int32, device="cuda"), torch.empty(2, 5, dtype=torch.int32, device="cuda")
    ws_s = torch.empty(binding.fa2_select_workspace_size(2, 5, c.wide), dtype=torch.uint8, device="cuda")
    ws = torch.empty(binding.fa2_decode_workspace_size(2, 15, 5, 72), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(2, 15, device="cuda")

    def step():
        binding.fa2_select_pages(q, bounds.t, exps.t, c.table_dev, c.lens_dev, sel, sel_lens, ws_s, 16)
        binding.fa2_decode_selected(q, *c.pools(), o, lse, sel, sel_lens, ws, 1 / math.sqrt(72))

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    torch.cuda.synchronize()
    got = o.clone(), lse.clone(), sel.clone()
    step()
    binding.fa2_device_status()
    assert torch.equal(got[0], o) and torch.equal(got[1], lse) and torch.equal(got[2], sel)
