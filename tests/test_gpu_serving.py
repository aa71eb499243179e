"""Rotary positions, the cache and the attention run together, as a program that generates tokens uses them."""
import math

import numpy as np
import pytest

from attention_fa2_forward_02_gb300 import binding, synth
from oracle import attention as A
from oracle import serving as S
from tests import gpu_util as G
from tests.paged import Cache
from tests.tolerance import UNIT_ROUNDOFF

pytestmark = pytest.mark.gpu

HKV, GROUP, D, PAGE = 2, 3, 64, 16
HEADS = HKV * GROUP


class Server:
    """Prompts of given lengths, then tokens one by one: the projections are seeded, everything after them the library's."""

    def __init__(self, prompts, steps, e4m3):
        torch = G.require_gpu()
        self.prompts, self.steps, self.e4m3 = prompts, steps, e4m3
        self.total = [n + steps for n in prompts]
        self.cache = Cache("server", self.total, PAGE, HKV, D, "bf16", e4m3, stale="nan")
        self.lens = torch.zeros(len(prompts), dtype=torch.int32, device="cuda")
        freq, self.magnitude = binding.fa2_rope_frequencies(D, 10000.0, "ramp", 4.0, 32.0)
        self.freq64, self.freq = freq.numpy(), freq.cuda()
        # all tokens of all sequences: q, k, v heads side by side
        self.qkv = [synth.tensor(f"server/{b}", (n, HEADS + 2 * HKV, D), "bf16") for b, n in enumerate(self.total)]
        self.ws = torch.empty(binding.fa2_decode_workspace_size(len(prompts), HEADS, HKV, D), dtype=torch.uint8, device="cuda")
        self.o = G.empty((len(prompts), HEADS, D), "bf16")
        self.lse = torch.empty(len(prompts), HEADS, device="cuda")

    def rotate(self, rows, positions):
        """q and k heads of rows [T, heads, D] turned in place."""
        view = rows[:, :HEADS + HKV].unsqueeze(0).transpose(1, 2)
        binding.fa2_rope(view, view, self.freq, positions=positions.unsqueeze(0), magnitude=self.magnitude)

    def prefill(self):
        torch = G.require_gpu()
        rows = torch.cat([G.to_device(x[:n], "bf16") for x, n in zip(self.qkv, self.prompts)])
        pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in self.prompts]).cuda()
        cu = torch.tensor(np.concatenate([[0], np.cumsum(self.prompts)]), dtype=torch.int32, device="cuda")
        self.lens.copy_(torch.tensor(self.prompts, dtype=torch.int32))
        self.rotate(rows, pos)
        self.store(rows, cu)

    def store(self, rows, cu=None):
        c = self.cache
        binding.fa2_kv_append(*c.pools(), rows[:, HEADS:HEADS + HKV], rows[:, HEADS + HKV:], c.table_dev, self.lens, cu_new=cu, **c.exps())

    def step(self, rows):
        """rows [batch, heads, D]: the new tokens' projections; lens already counts them in."""
        c = self.cache
        self.rotate(rows, self.lens - 1)
        self.store(rows)
        binding.fa2_decode(rows[:, :HEADS], *c.pools(), self.o, self.lse, c.table_dev, self.lens, self.ws, 1 / math.sqrt(D), **c.exps())

    def new_rows(self, i):
        return np.stack([x[n + i] for x, n in zip(self.qkv, self.prompts)])

    def reference(self, i):
        """O after step i from the unquantised float64 projections."""
        out = []
        for x, n in zip(self.qkv, self.prompts):
            w = synth.widen(x[: n + i + 1], "bf16")
            t = S.rope(w[:, :HEADS + HKV].swapaxes(0, 1)[None], np.arange(n + i + 1)[None], self.freq64, False, self.magnitude)[0]
            k, v = t[HEADS:], w[:, HEADS + HKV:].swapaxes(0, 1)
            q = t[:HEADS, -1].reshape(HKV, GROUP, D)
            out.append(A.forward(q, k, v, 1 / math.sqrt(D))[0].reshape(HEADS, D))
        return np.stack(out)


def tolerance(e4m3):
    """q and k rounded to bfloat16 after the rotation (2^-8 each) and, with e4m3, k and v by 2^-4: a score of |s| <= E then
    moves by about sqrt(d) roundings of its terms, not d; with unit normal rows and scale 1 / sqrt(d), its terms' root sum of
    squares is about 1, so a score moves by 8 * 2^-4 at 8 of Hoeffding's deviations (8 * 2^-7 without e4m3), every weight by the
    factor exp of that, and O, an average of unit values of at most about 4, by twice that times 4 at the very most."""
    return 2 * 4 * math.expm1(8 * (2.0 ** -4 if e4m3 else 2.0 ** -7)) / 2 ** 2


@pytest.mark.parametrize("e4m3", [False, True])
def test_generation_follows_the_oracle(e4m3):
    s = Server([33, 1, 64, 17], 20, e4m3)
    s.prefill()
    for i in range(s.steps):
        s.lens += 1
        s.step(G.to_device(s.new_rows(i), "bf16"))
        binding.fa2_device_status()
        ref = s.reference(i)
        err = G.to_f64(s.o) - ref
        assert np.max(np.abs(err)) <= tolerance(e4m3)
        # a wrong position, page or head makes an error as large as the result itself
        assert np.sqrt(np.mean(err ** 2)) <= (0.15 if e4m3 else 0.02) * np.sqrt(np.mean(ref ** 2))


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_captured_step_replays_with_new_lengths(e4m3):
    """One graph of (length + 1, rotate, store, attend) replayed for every token gives what the eager calls give."""
    torch = G.require_gpu()
    a, b = (Server([33, 1, 64, 17], 20, e4m3) for _ in range(2))
    a.prefill()
    b.prefill()
    rows = torch.empty(4, HEADS + 2 * HKV, D, dtype=torch.bfloat16, device="cuda")

    def one():
        b.lens += 1
        b.step(rows)

    keep = [t.clone() for t in (b.lens, *[p.view(torch.uint8) for p in b.cache.pools()])]
    rows.copy_(G.to_device(b.new_rows(0), "bf16"))
    one()  # eager once, for the library's one-time settings
    torch.cuda.synchronize()
    b.lens.copy_(keep[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    b.lens.copy_(keep[0])
    for i in range(a.steps):
        a.lens += 1
        a.step(G.to_device(a.new_rows(i), "bf16"))
        rows.copy_(G.to_device(b.new_rows(i), "bf16"))
        b.o.fill_(float("nan"))
        graph.replay()
        assert torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse), f"token {i}"
    for x, y in zip(a.cache.pools(), b.cache.pools()):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("e4m3", [False, True])
def test_read_back_feeds_the_forward(e4m3):
    """The cache read back, its heads' grouped queries as query rows: fa2_forward and fa2_decode agree."""
    torch = G.require_gpu()
    n, batch = 300, 3
    c = Cache("feed", [n] * batch, PAGE, HKV, D, "bf16", e4m3)
    q = G.to_device(synth.tensor("feed/q", (batch, HEADS, D), "bf16"), "bf16")
    o, lse = torch.empty_like(q), torch.empty(batch, HEADS, device="cuda")
    ws = torch.empty(binding.fa2_decode_workspace_size(batch, HEADS, HKV, D), dtype=torch.uint8, device="cuda")
    binding.fa2_decode(q, *c.pools(), o, lse, c.table_dev, c.lens_dev, ws, 0.125, **c.exps())
    k, v = (G.empty((batch, HKV, n, D), "bf16") for _ in "kv")
    binding.fa2_kv_read(*c.pools(), k, v, c.table_dev, c.lens_dev, **c.exps())
    rows = batch * HKV
    o2, lse2 = torch.empty_like(q).view(rows, GROUP, D), torch.empty(rows, GROUP, device="cuda")
    binding.fa2_forward(q.view(rows, GROUP, D), k.view(rows, n, D), v.view(rows, n, D), o2, lse2, 0.125)
    binding.fa2_device_status()
    a, b = G.to_f64(o).reshape(rows, GROUP, D), G.to_f64(o2)
    v64 = np.abs(G.to_f64(v)).reshape(rows, 1, n, D).max(2)
    # both are within two roundings of 2^-8 (weights, output) of sum P |v| <= max |v|
    assert np.all(np.abs(a - b) <= 4 * UNIT_ROUNDOFF["bf16"] * v64 + 1e-5)
    assert np.max(np.abs(G.to_f64(lse).reshape(rows, GROUP) - G.to_f64(lse2))) <= 2e-4


SCRIPT = """
import math, sys
import torch
from attention_fa2_forward_02_gb300 import binding as B

def attention():
    for d in (32, 64, 128):
        for dt in (torch.bfloat16, torch.float16):
            for bh, n_q, n_k in ((2, 4096, 128), (2, 200, 2048), (80, 200, 300)):
                q, o, do, dq = (torch.randn(bh, n_q, d, device="cuda").to(dt) for _ in range(4))
                k, v, dk, dv = (torch.randn(bh, n_k, d, device="cuda").to(dt) for _ in range(4))
                lse = torch.empty(bh, n_q, device="cuda")
                B.fa2_forward(q, k, v, o, lse, 0.2)
                ws = torch.empty(B.fa2_backward_workspace_size(bh, n_q, n_k, d, B._dtype_code(q)), dtype=torch.uint8, device="cuda")
                B.fa2_backward(q, k, v, o, do, lse, dq, dk, dv, ws, 0.2)

def decode():
    table, lens = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4), torch.tensor([60, 33], dtype=torch.int32, device="cuda")
    for d in (32, 64, 128):
        for dt in (torch.bfloat16, torch.float16):
            for group in (2, 16):
                pages = torch.randn(8, 2, 16, d, device="cuda").to(dt)
                exp = torch.full((8, 2, 16), 127, dtype=torch.uint8, device="cuda")
                q = torch.randn(2, 2 * group, d, device="cuda").to(dt)
                o, lse = torch.empty_like(q), torch.empty(2, 2 * group, device="cuda")
                ws = torch.empty(B.fa2_decode_workspace_size(2, 2 * group, 2, d), dtype=torch.uint8, device="cuda")
                B.fa2_decode(q, pages, pages, o, lse, table, lens, ws, 0.2)
                codes = pages.to(torch.float8_e4m3fn)
                B.fa2_decode(q, codes, codes, o, lse, table, lens, ws, 0.2, k_exp=exp, v_exp=exp)

for name in sys.argv[1:]:
    {"attention": attention, "decode": decode}[name]()
    B.fa2_device_status()
"""


@pytest.mark.parametrize("order", [("attention", "decode"), ("decode", "attention")])
def test_both_orders_beside_the_attention_kernels(order):
    """Every kernel raises its own shared-memory limit, whatever ran before it in a fresh process."""
    import os
    import subprocess
    import sys
    G.require_gpu()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SCRIPT, *order], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-2000:]


CAPTURE_FIRST = """
import torch
from attention_fa2_forward_02_gb300 import binding as B
pages = torch.randn(8, 2, 16, 64, device="cuda").bfloat16()
table, lens = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4), torch.tensor([60, 33], dtype=torch.int32, device="cuda")
f = torch.ones(32, dtype=torch.float64, device="cuda")

def run():
    q = torch.ones(2, 4, 64, device="cuda").bfloat16()
    k, out = torch.ones(2, 2, 64, device="cuda").bfloat16(), [torch.zeros(2, 2, 64, 64, device="cuda").bfloat16() for _ in "kv"]
    o, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    ws = torch.empty(B.fa2_decode_workspace_size(2, 4, 2, 64), dtype=torch.uint8, device="cuda")
    B.fa2_rope(q.unsqueeze(2), q.unsqueeze(2), f)
    B.fa2_kv_append(pages, pages.clone(), k, k, table, lens)
    B.fa2_decode(q, pages, pages, o, lse, table, lens, ws, 0.2)
    B.fa2_kv_read(pages, pages, *out, table, lens)
    return o, lse, *out

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
want = run()
B.fa2_device_status()
assert all(torch.equal(a, b) for a, b in zip(got, want))
"""


def test_the_first_calls_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    G.require_gpu()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE_FIRST], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("threads", [4])
def test_calls_from_several_host_threads(threads):
    """Threads with streams and workspaces of their own get what one call alone gets."""
    import threading
    torch = G.require_gpu()
    c = Cache("threads", [700, 33, 1500], PAGE, HKV, D, "bf16", True)
    q = G.to_device(synth.tensor("threads/q", (3, HEADS, D), "bf16"), "bf16")

    def call(stream=None):
        o, lse = torch.empty_like(q), torch.empty(3, HEADS, device="cuda")
        ws = torch.empty(binding.fa2_decode_workspace_size(3, HEADS, HKV, D), dtype=torch.uint8, device="cuda")
        k, v = (torch.zeros(3, HKV, 1500, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        torch.cuda.synchronize()
        for _ in range(20):
            binding.fa2_decode(q, *c.pools(), o, lse, c.table_dev, c.lens_dev, ws, 0.125, stream=stream, **c.exps())
            binding.fa2_kv_read(*c.pools(), k, v, c.table_dev, c.lens_dev, stream=stream, **c.exps())
        torch.cuda.synchronize()
        return o, lse, k, v

    want, got = call(), [None] * threads

    def work(i):
        got[i] = call(torch.cuda.Stream())

    ts = [threading.Thread(target=work, args=(i,)) for i in range(threads)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    for g in got:
        assert g is not None and all(torch.equal(a, b) for a, b in zip(g, want))
