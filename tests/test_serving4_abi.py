"""Refusals of the rotated append, the 4-bit cache, the bounds, the selection and its attention: on the host, before anything is
launched (no GPU needed)."""
import ctypes

import pytest

from attention_fa2_forward_02_gb300 import binding
from attention_fa2_forward_02_gb300 import build as build_mod
from tests.test_serving_abi import (BF16, CACHE_REFUSALS, F32, INVALID, MISALIGNED, ODD, P, PM, UNSUPPORTED, WORKSPACE, append, cache,
                                    decode, i64, read)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return binding.library()


def cache4(**kw):
    """4-bit pages; strides count elements."""
    return cache(**({"type": 2, "k_exp": 0x1000, "v_exp": 0x1000, "k_scale": 0x1000, "v_scale": 0x1000} | kw))


@pytest.mark.parametrize("call", [append, read, decode])
@pytest.mark.parametrize("kw,want", [
    ({"k_exp": None}, INVALID), ({"v_exp": None}, INVALID), ({"k_scale": None}, INVALID), ({"v_scale": None}, INVALID), ({"type": 3}, INVALID),
    ({"head_dim": 48}, UNSUPPORTED), ({"head_dim": 16}, UNSUPPORTED), ({"head_dim": 160, "slot_stride": 160, "head_stride": 2560, "page_stride": 10240},
                                                                       UNSUPPORTED),
    ({"k_exp": 0x1008}, MISALIGNED), ({"v_exp": 0x1001}, MISALIGNED), ({"k_scale": 0x1008}, MISALIGNED), ({"v_scale": 0x1001}, MISALIGNED), ({"k": 0x1008}, MISALIGNED),
    ({"slot_stride": 80, "head_stride": 16 * 80, "page_stride": 64 * 80}, MISALIGNED), ({"slot_stride": 32}, INVALID),
])
def test_four_bit_cache_validation(lib, call, kw, want):
    assert call(lib, cache4(**kw)) == want


def rope_append(lib, c=None, q=P, qo=P, k=P, v=P, qs=(512, 64), os=(512, 64), ks=(512, 64), vs=(512, 64), f=P, rot=64, mag=1.0, pos=P, table=P, ts=8,
                pages=8, cu=P, lens=P, batch=3, tokens=9, heads=8, dt=BF16):
    c = c or cache()
    st = lambda s: None if s is None else i64(*s)  # noqa: E731
    return lib.fa2_rope_append(ctypes.byref(c), q, qo, k, v, st(qs), st(os), st(ks), st(vs), f, rot, 0, mag, pos, table, ts, pages, cu, lens, batch, tokens,
                               heads, dt, None)


def bounds(lib, c=None, b=P, e=P, table=P, ts=8, pages=8, cu=P, lens=P, batch=3, tokens=9, dt=BF16):
    c = c or cache()
    return lib.fa2_kv_bounds(ctypes.byref(c), b, e, table, ts, pages, cu, lens, batch, tokens, dt, None)


def selected(lib, c=None, q=P, qs=(512, 64), o=P, lse=P, table=P, pages=8, lens=P, batch=3, heads=8, ws=P, wsb=1 << 24, dt=BF16, scale=0.125):
    c = c or cache()
    return lib.fa2_decode_selected(q, i64(*qs), ctypes.byref(c), o, lse, table, pages, lens, batch, heads, ws, wsb, dt, scale, None)


def select(lib, q=P, qs=(512, 64), b=P, e=P, n=10, page=16, heads=8, hkv=4, d=64, table=P, ts=8, pages=8, lens=P, batch=3, sel=P, sl=P, budget=4, first=1,
           recent=1, ws=P, wsb=1 << 20, dt=BF16):
    return lib.fa2_select_pages(q, i64(*qs), b, e, n, page, heads, hkv, d, table, ts, pages, lens, batch, sel, sl, budget, first, recent, ws, wsb, dt, None)


@pytest.mark.parametrize("call", [rope_append, selected])
@pytest.mark.parametrize("kw,want", CACHE_REFUSALS)
def test_cache_validation(lib, call, kw, want):
    assert call(lib, cache(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    ({"q": None}, INVALID), ({"qo": None}, INVALID), ({"q": None, "qo": None}, INVALID), ({"heads": 0}, INVALID), ({"heads": -1}, INVALID),
    ({"qs": None}, INVALID), ({"os": None}, INVALID), ({"k": None}, INVALID), ({"v": None}, INVALID), ({"ks": None}, INVALID), ({"f": None}, INVALID),
    ({"rot": 0}, INVALID), ({"rot": 17}, INVALID), ({"rot": 80}, INVALID), ({"rot": 24}, UNSUPPORTED), ({"mag": float("nan")}, INVALID),
    ({"mag": float("inf")}, INVALID), ({"tokens": 0}, INVALID), ({"cu": None}, INVALID), ({"os": (512, 32)}, INVALID), ({"os": (256, 64)}, INVALID),
    ({"os": (1024, 64)}, INVALID),  # q_out is q, with other strides
    ({"qs": (-512, 64), "os": (-512, 64)}, INVALID), ({"heads": 65536, "qs": (1 << 23, 64), "os": (1 << 23, 64)}, UNSUPPORTED),
    ({"dt": F32}, UNSUPPORTED), ({"dt": 7}, INVALID), ({"tokens": 1 << 31}, UNSUPPORTED), ({"q": PM}, MISALIGNED), ({"qo": PM}, MISALIGNED),
    ({"k": PM}, MISALIGNED), ({"f": ctypes.c_void_p(0x1004)}, MISALIGNED), ({"pos": ODD}, MISALIGNED), ({"cu": ODD}, MISALIGNED),
    ({"qs": (516, 64), "qo": ctypes.c_void_p(0x2000)}, MISALIGNED), ({"os": (1024, 68), "qo": ctypes.c_void_p(0x2000)}, MISALIGNED), ({"table": None}, INVALID), ({"ts": 7}, INVALID),
])
def test_rope_append_validation(lib, kw, want):
    assert rope_append(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    ({"b": None}, INVALID), ({"e": None}, INVALID), ({"tokens": 0}, INVALID), ({"cu": None}, INVALID), ({"table": None}, INVALID), ({"lens": None}, INVALID),
    ({"batch": 0}, INVALID), ({"batch": 65536, "tokens": 1 << 20}, UNSUPPORTED), ({"tokens": 1 << 31}, UNSUPPORTED), ({"dt": F32}, UNSUPPORTED),
    ({"b": PM}, MISALIGNED), ({"cu": ODD}, MISALIGNED), ({"table": ODD}, MISALIGNED),
])
def test_bounds_validation(lib, kw, want):
    assert bounds(lib, **kw) == want


def test_bounds_want_keys_alone(lib):
    """Everything but the bounds' own alignment is in order without values."""
    assert bounds(lib, cache(v=None), b=PM) == MISALIGNED and bounds(lib, cache4(v=None, v_exp=None, v_scale=None), b=PM) == MISALIGNED
    assert bounds(lib, cache(k=None), b=PM) == INVALID and bounds(lib, cache4(k_scale=None), b=PM) == INVALID


@pytest.mark.parametrize("kw,want", [
    ({"q": None}, INVALID), ({"b": None}, INVALID), ({"e": None}, INVALID), ({"table": None}, INVALID), ({"lens": None}, INVALID), ({"sel": None}, INVALID),
    ({"sl": None}, INVALID), ({"n": 0}, INVALID), ({"page": 0}, INVALID), ({"heads": 0}, INVALID), ({"heads": 6}, INVALID), ({"hkv": 0}, INVALID),
    ({"d": 0}, INVALID), ({"batch": 0}, INVALID), ({"pages": 0}, INVALID), ({"ts": 7}, INVALID), ({"ts": -1}, INVALID), ({"budget": 0}, INVALID),
    ({"first": -1}, INVALID), ({"recent": -1}, INVALID), ({"first": 5, "recent": 0}, INVALID), ({"first": 2, "recent": 3}, INVALID), ({"qs": (-512, 64)}, INVALID),
    ({"dt": 4}, INVALID), ({"dt": F32}, UNSUPPORTED), ({"d": 60}, UNSUPPORTED), ({"d": 136}, UNSUPPORTED), ({"heads": 516, "qs": (1 << 20, 64)}, UNSUPPORTED),
    ({"hkv": 1025, "heads": 1025}, UNSUPPORTED), ({"batch": 65536}, UNSUPPORTED), ({"n": 1 << 31}, UNSUPPORTED), ({"pages": 1 << 27, "ts": 1 << 27}, UNSUPPORTED),
    ({"budget": 1 << 27}, UNSUPPORTED), ({"batch": 65535, "hkv": 32, "heads": 32}, UNSUPPORTED), ({"q": PM}, MISALIGNED), ({"b": PM}, MISALIGNED),
    ({"table": ODD}, MISALIGNED), ({"lens": ODD}, MISALIGNED), ({"sel": ODD}, MISALIGNED), ({"sl": ODD}, MISALIGNED), ({"qs": (516, 64)}, MISALIGNED),
    ({"ws": None}, WORKSPACE), ({"ws": PM}, WORKSPACE), ({"wsb": 3 * 4 * 8 * 4 - 1}, WORKSPACE),
])
def test_select_validation(lib, kw, want):
    assert select(lib, **kw) == want


def test_select_workspace_size(lib):
    size = lib.fa2_select_workspace_size
    assert size(3, 4, 8) == 3 * 4 * 8 * 4
    for bad in ((0, 4, 8), (3, 0, 8), (3, 4, 0), (65536, 4, 8), (3, 1025, 8), (3, 4, (1 << 30) + 1)):
        assert size(*bad) == 0


@pytest.mark.parametrize("kw,want", [
    ({"q": None}, INVALID), ({"o": None}, INVALID), ({"lse": None}, INVALID), ({"table": None}, INVALID), ({"lens": None}, INVALID), ({"pages": 0}, INVALID),
    ({"heads": 6}, INVALID), ({"scale": 0.0}, INVALID), ({"q": PM}, MISALIGNED), ({"ws": None}, WORKSPACE), ({"wsb": 1000}, WORKSPACE),
    ({"batch": 65536}, UNSUPPORTED), ({"pages": 1 << 27}, UNSUPPORTED),
])
def test_selected_validation(lib, kw, want):
    assert selected(lib, **kw) == want


def test_selected_heads_of_all_sequences(lib):
    c = cache(n_kv_heads=1024, page_stride=1024 * 1024)
    assert selected(lib, c, batch=1025, heads=1024) == UNSUPPORTED


def test_binding_refusals():
    """Shapes, types and devices, before any library call."""
    torch = pytest.importorskip("torch")
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i32, u8, f8 = torch.int32, torch.uint8, torch.float8_e4m3fn
    pages, table, lens, rows = z(6, 2, 16, 32), z(3, 2, dt=i32), z(3, dt=i32), z(3, 2, 64)
    four = {"k_pages": z(6, 2, 16, 32, dt=u8), "v_pages": z(6, 2, 16, 32, dt=u8)}
    scales = {"k_exp": z(6, 2, 16, dt=u8), "v_exp": z(6, 2, 16, dt=u8), "k_scale": z(6, 2, 16, 4).to(f8), "v_scale": z(6, 2, 16, 4).to(f8)}
    good = four | scales | {"k": rows, "v": rows, "block_table": table, "seq_lens": lens}
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.fa2_kv_append(**good)
    for bad in ({"k_exp": None}, {"k_scale": None}, {"v_scale": z(6, 2, 16, 2).to(f8)}, {"k": z(3, 2, 32), "v": z(3, 2, 32)},
                {"k_pages": z(6, 2, 16, 64), "v_pages": z(6, 2, 16, 64), "k_exp": None, "v_exp": None}):
        with pytest.raises(ValueError):
            binding.fa2_kv_append(**(good | bad))
    for bad in ({"k_scale": z(6, 2, 16, 4, dt=u8)}, {"v_exp": z(6, 2, 16)}):
        with pytest.raises(TypeError):
            binding.fa2_kv_append(**(good | bad))

    freq, rows = torch.ones(16, dtype=torch.float64), z(3, 2, 32)
    q = z(3, 4, 32)
    good = {"k_pages": pages, "v_pages": pages, "k": rows, "v": rows, "inv_freq": freq, "block_table": table, "seq_lens": lens, "q": q, "q_out": q}
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.fa2_rope_append(**good)
    for bad in ({"q": None}, {"q_out": None}, {"q_out": z(3, 2, 32)}, {"q": z(2, 4, 32), "q_out": z(2, 4, 32)}, {"positions": z(4, dt=i32)},
                {"cu_new": z(3, dt=i32)}, {"k": z(3, 3, 32), "v": z(3, 3, 32)}, {"inv_freq": freq[None]}):
        with pytest.raises(ValueError):
            binding.fa2_rope_append(**(good | bad))
    for bad in ({"q": q.half(), "q_out": q.half()}, {"q_out": q.half()}, {"inv_freq": freq.float()}, {"positions": z(3, dt=torch.int64)}, {"v": rows.half()}):
        with pytest.raises(TypeError):
            binding.fa2_rope_append(**(good | bad))

    b, e = z(6, 2, 2, 32, dt=torch.int8), z(6, 2, dt=u8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.fa2_kv_bounds(pages, b, e, table, lens, 3)
    for bad in ({"bounds": b[:5]}, {"bounds_exp": e[:5]}, {"cu_new": z(3, dt=i32)}, {"k_exp": e}):
        with pytest.raises(ValueError):
            binding.fa2_kv_bounds(**({"k_pages": pages, "bounds": b, "bounds_exp": e, "block_table": table, "seq_lens": lens, "tokens": 3} | bad))
    with pytest.raises(TypeError):
        binding.fa2_kv_bounds(pages, b.view(u8), e, table, lens, 3)
    with pytest.raises(TypeError):
        binding.fa2_kv_bounds(z(6, 2, 16, 32, dt=torch.float32), b, e, table, lens, 3)

    sel, sl, ws = z(3, 2, 4, dt=i32), z(3, 2, dt=i32), z(64, dt=u8)
    good = {"q": q, "bounds": b, "bounds_exp": e, "block_table": table, "seq_lens": lens, "sel_table": sel, "sel_lens": sl, "workspace": ws, "page_size": 16}
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.fa2_select_pages(**good)
    for bad in ({"q": z(3, 4, 16)}, {"q": z(2, 4, 32)}, {"bounds": b[0]}, {"bounds_exp": e[:5]}, {"sel_table": z(3, 4, 4, dt=i32)}, {"sel_lens": z(3, dt=i32)},
                {"seq_lens": z(2, dt=i32)}, {"page_size": -1}):
        with pytest.raises(ValueError):
            binding.fa2_select_pages(**(good | bad))
    for bad in ({"bounds": b.float()}, {"sel_table": sel.long()}, {"block_table": table.long()}, {"q": q.double()}):
        with pytest.raises(TypeError):
            binding.fa2_select_pages(**(good | bad))

    lse = z(3, 4, dt=torch.float32)
    good = {"q": q, "k_pages": pages, "v_pages": pages, "o": q, "lse": lse, "sel_table": sel, "sel_lens": sl, "workspace": ws, "softmax_scale": 0.2}
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.fa2_decode_selected(**good)
    for bad in ({"sel_table": table}, {"sel_table": z(3, 4, 4, dt=i32)}, {"sel_lens": lens}):
        with pytest.raises(ValueError):
            binding.fa2_decode_selected(**(good | bad))
