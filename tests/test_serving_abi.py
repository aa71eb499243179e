"""Refusals of the rotary, cache and decode calls: on the host, before anything is launched (no GPU needed)."""
import ctypes

import pytest

from attention_fa2_forward_02_gb300 import binding
from attention_fa2_forward_02_gb300 import build as build_mod

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA_ERR, TIMEOUT, WORKSPACE = range(7)
F32, F16, BF16 = 0, 1, 2
P = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation first
PM = ctypes.c_void_p(0x1008)
ODD = ctypes.c_void_p(0x1002)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return binding.library()


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def rope(lib, x=P, y=P, pos=P, ps=0, f=P, b=2, h=3, n=5, d=64, rot=64, xs=(960, 320, 64), ys=(960, 320, 64), mag=1.0, dt=BF16,
         back=False):
    fn = lib.fa2_rope_backward if back else lib.fa2_rope
    return fn(x, y, pos, ps, f, b, h, n, d, rot, None if xs is None else i64(*xs), None if ys is None else i64(*ys), 0, mag, dt, None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,want", [
    ({"x": None}, INVALID), ({"y": None}, INVALID), ({"f": None}, INVALID), ({"xs": None}, INVALID), ({"b": 0}, INVALID),
    ({"h": -1}, INVALID), ({"n": 0}, INVALID), ({"d": 0}, INVALID), ({"rot": 0}, INVALID), ({"rot": 33}, INVALID),
    ({"rot": 66}, INVALID), ({"dt": 5}, INVALID), ({"mag": float("nan")}, INVALID), ({"mag": float("inf")}, INVALID),
    ({"ps": -1}, INVALID), ({"xs": (-960, 320, 64)}, INVALID), ({"ys": (960, 320, 0)}, INVALID),
    ({"ys": (960, 320, 63)}, INVALID), ({"ys": (960, 0, 64)}, INVALID), ({"ys": (640, 320, 64)}, INVALID),
    ({"xs": (0, 320, 64)}, INVALID),  # y is x, with other strides
    ({"d": 1025, "rot": 64, "xs": (1 << 20, 1 << 15, 2048), "ys": (1 << 20, 1 << 15, 2048)}, UNSUPPORTED),
    ({"n": (1 << 30) + 1, "h": 1, "b": 1}, UNSUPPORTED), ({"b": 1 << 20, "h": 1 << 12}, UNSUPPORTED),
    ({"x": PM}, MISALIGNED), ({"y": PM, "x": P}, MISALIGNED), ({"f": ctypes.c_void_p(0x1004)}, MISALIGNED), ({"pos": ODD}, MISALIGNED),
])
def test_rope_validation(lib, back, kw, want):
    assert rope(lib, back=back, **kw) == want


def cache(**kw):
    c = binding.KvCache()
    c.k, c.v, c.k_exp, c.v_exp = 0x1000, 0x1000, 0, 0
    c.num_pages, c.n_kv_heads, c.page_size, c.head_dim, c.type = 10, 4, 16, 64, 0
    c.page_stride, c.head_stride, c.slot_stride = 4 * 16 * 64, 16 * 64, 64
    for k, v in kw.items():
        setattr(c, k, v)
    return c


CACHE_REFUSALS = [
    ({"k": None}, INVALID), ({"v": None}, INVALID), ({"type": 2}, INVALID), ({"type": 1}, INVALID), ({"num_pages": 0}, INVALID),
    ({"n_kv_heads": 0}, INVALID), ({"page_size": 0}, INVALID), ({"head_dim": 0}, INVALID), ({"page_stride": -4096}, INVALID),
    ({"slot_stride": 32}, INVALID), ({"head_stride": 0}, INVALID), ({"page_stride": 1024}, INVALID),
    ({"head_dim": 60}, UNSUPPORTED), ({"head_dim": 136, "slot_stride": 136, "head_stride": 2176, "page_stride": 8704}, UNSUPPORTED),
    ({"type": 1, "k_exp": 0x1001, "v_exp": 0x1001, "head_dim": 56}, UNSUPPORTED),
    ({"k": 0x1008}, MISALIGNED), ({"v": 0x1002}, MISALIGNED),
    ({"slot_stride": 68, "head_stride": 16 * 68, "page_stride": 64 * 68}, MISALIGNED),
    ({"type": 1, "k_exp": 0x1001, "v_exp": 0x1001, "slot_stride": 72, "head_stride": 16 * 72, "page_stride": 64 * 72}, MISALIGNED),
    ({"num_pages": 1 << 31}, UNSUPPORTED),
    ({"n_kv_heads": 1025, "page_stride": 1025 * 1024}, UNSUPPORTED),
]


def append(lib, c=None, k=P, v=P, ks=(512, 64), vs=(512, 64), table=P, ts=8, pages=8, cu=P, lens=P, batch=3, tokens=9, dt=BF16):
    c = c or cache()
    return lib.fa2_kv_append(ctypes.byref(c), k, v, i64(*ks), i64(*vs), table, ts, pages, cu, lens, batch, tokens, dt, None)


def read(lib, c=None, k=P, v=P, os=(4 * 40 * 64, 40 * 64, 64), table=P, ts=8, pages=8, lens=P, batch=3, n=40, dt=BF16):
    c = c or cache()
    return lib.fa2_kv_read(ctypes.byref(c), k, v, i64(*os), table, ts, pages, lens, batch, n, dt, None)


def decode(lib, c=None, q=P, qs=(512, 64), o=P, lse=P, table=P, ts=8, pages=8, lens=P, batch=3, heads=8, window=0, ws=P,
           wsb=1 << 24, dt=BF16, scale=0.125):
    c = c or cache()
    return lib.fa2_decode(q, i64(*qs), ctypes.byref(c), o, lse, table, ts, pages, lens, batch, heads, window, ws, wsb, dt, scale, None)


@pytest.mark.parametrize("call", [append, read, decode])
@pytest.mark.parametrize("kw,want", CACHE_REFUSALS)
def test_cache_validation(lib, call, kw, want):
    assert call(lib, cache(**kw)) == want


@pytest.mark.parametrize("call", [append, read, decode])
@pytest.mark.parametrize("kw,want", [
    ({"table": None}, INVALID), ({"lens": None}, INVALID), ({"batch": 0}, INVALID), ({"pages": 0}, INVALID), ({"ts": 7}, INVALID),
    ({"ts": -1}, INVALID), ({"dt": 9}, INVALID), ({"dt": F32}, UNSUPPORTED), ({"batch": 65536, "cu": P}, UNSUPPORTED),
    ({"pages": 1 << 27, "ts": 1 << 27}, UNSUPPORTED), ({"table": ODD}, MISALIGNED), ({"lens": ODD}, MISALIGNED),
])
def test_table_validation(lib, call, kw, want):
    if call is not append:
        kw.pop("cu", None)
    assert call(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    ({"k": None}, INVALID), ({"v": None}, INVALID), ({"tokens": 0}, INVALID), ({"cu": None}, INVALID),  # 9 rows, 3 sequences
    ({"ks": (-512, 64)}, INVALID), ({"tokens": 1 << 31}, UNSUPPORTED), ({"k": PM}, MISALIGNED), ({"cu": ODD}, MISALIGNED),
    ({"ks": (516, 64)}, MISALIGNED), ({"vs": (512, 68)}, MISALIGNED),
])
def test_append_validation(lib, kw, want):
    assert append(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    ({"k": None}, INVALID), ({"v": None}, INVALID), ({"n": 0}, INVALID), ({"os": (0, 2560, 64)}, INVALID),
    ({"os": (10240, 2560, 56)}, INVALID), ({"os": (-10240, 2560, 64)}, INVALID), ({"n": (1 << 30) + 1}, UNSUPPORTED),
    ({"k": PM}, MISALIGNED), ({"os": (4 * 40 * 68, 40 * 68, 68)}, MISALIGNED),
])
def test_read_validation(lib, kw, want):
    assert read(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    ({"q": None}, INVALID), ({"o": None}, INVALID), ({"lse": None}, INVALID), ({"heads": 0}, INVALID), ({"heads": 6}, INVALID),
    ({"window": -1}, INVALID), ({"scale": 0.0}, INVALID), ({"scale": float("nan")}, INVALID), ({"scale": float("inf")}, INVALID),
    ({"qs": (-512, 64)}, INVALID), ({"heads": 65536}, UNSUPPORTED), ({"q": PM}, MISALIGNED), ({"o": PM}, MISALIGNED),
    ({"lse": PM}, MISALIGNED), ({"qs": (512, 60)}, MISALIGNED), ({"ws": None}, WORKSPACE), ({"ws": PM}, WORKSPACE), ({"wsb": 1000}, WORKSPACE),
])
def test_decode_validation(lib, kw, want):
    assert decode(lib, **kw) == want


def test_decode_workspace_size(lib):
    size = lib.fa2_decode_workspace_size
    assert 0 < size(1, 32, 8, 128) <= 16 << 20 and size(1, 8, 8, 64) < size(1, 8, 8, 128)
    for bad in ((0, 8, 8, 64), (1, 0, 8, 64), (1, 8, 0, 64), (1, 8, 3, 64), (1, 8, 8, 0), (1, 8, 8, 60), (1, 8, 8, 136)):
        assert size(*bad) == 0


def test_binding_refusals():
    """Shapes, types and devices, before any library call: CPU tensors pass these checks only to be refused as such."""
    torch = pytest.importorskip("torch")
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    f, i32 = torch.ones(16, dtype=torch.float64), torch.int32
    x = z(1, 2, 5, 32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.fa2_rope(x, x, f)
    with pytest.raises(ValueError):
        binding.fa2_rope(x[0], x[0], f)
    with pytest.raises(ValueError):
        binding.fa2_rope(x, z(1, 2, 6, 32), f)
    with pytest.raises(ValueError):
        binding.fa2_rope(x, x, f, positions=z(4, dt=i32))
    with pytest.raises(TypeError):
        binding.fa2_rope(x, x, f, positions=z(5, dt=torch.int64))
    with pytest.raises(TypeError):
        binding.fa2_rope_backward(x, x.half(), f)
    with pytest.raises(TypeError):
        binding.fa2_rope(x, x, f.float())

    pages, table, lens = z(6, 2, 16, 32), z(3, 2, dt=i32), z(3, dt=i32)
    rows, ws = z(3, 2, 32), z(64, dt=torch.uint8)
    exp = z(6, 2, 16, dt=torch.uint8)
    fp8 = pages.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.fa2_kv_append(pages, pages, rows, rows, table, lens)
    for bad in ({"k_pages": pages[0]}, {"v_pages": z(5, 2, 16, 32)}, {"v_pages": z(6, 16, 2, 32).transpose(1, 2)}, {"k": z(3, 4, 32)},
                {"v": z(2, 2, 32)}, {"block_table": z(3, dt=i32)}, {"seq_lens": z(2, dt=i32)}, {"cu_new": z(3, dt=i32)},
                {"k_exp": exp}, {"k_pages": fp8, "v_pages": fp8}, {"k_pages": fp8, "v_pages": fp8, "k_exp": exp, "v_exp": exp[:5]}):
        args = {"k_pages": pages, "v_pages": pages, "k": rows, "v": rows, "block_table": table, "seq_lens": lens} | bad
        with pytest.raises(ValueError):
            binding.fa2_kv_append(**args)
    for bad in ({"v": rows.half()}, {"k_pages": pages.half(), "v_pages": pages.half()}, {"block_table": table.long()},
                {"seq_lens": lens.long()}, {"cu_new": z(4, dt=torch.int64)},
                {"k_pages": fp8, "v_pages": fp8, "k_exp": exp, "v_exp": exp.float()}):
        args = {"k_pages": pages, "v_pages": pages, "k": rows, "v": rows, "block_table": table, "seq_lens": lens} | bad
        with pytest.raises(TypeError):
            binding.fa2_kv_append(**args)
    out = z(3, 2, 20, 32)
    for bad in ({"k_out": z(3, 2, 32)}, {"k_out": z(2, 2, 20, 32), "v_out": z(2, 2, 20, 32)}, {"v_out": z(3, 20, 2, 32).transpose(1, 2)}):
        with pytest.raises(ValueError):
            binding.fa2_kv_read(**({"k_pages": pages, "v_pages": pages, "k_out": out, "v_out": out, "block_table": table,
                                    "seq_lens": lens} | bad))
    with pytest.raises(TypeError):
        binding.fa2_kv_read(pages, pages, out, out.half(), table, lens)
    q, lse = z(3, 4, 32), z(3, 4, dt=torch.float32)
    for bad in ({"q": z(2, 4, 32), "o": z(2, 4, 32)}, {"o": z(3, 2, 32)}, {"lse": z(3, 2, dt=torch.float32)}, {"q": z(3, 4, 16)}):
        with pytest.raises(ValueError):
            binding.fa2_decode(**({"q": q, "k_pages": pages, "v_pages": pages, "o": q, "lse": lse, "block_table": table,
                                   "seq_lens": lens, "workspace": ws, "softmax_scale": 0.2} | bad))
    with pytest.raises(TypeError):
        binding.fa2_decode(q, pages, pages, q, lse.half(), table, lens, ws, 0.2)
    with pytest.raises(TypeError):
        binding.fa2_decode(q, pages, pages, q.half(), lse, table, lens, ws, 0.2)
