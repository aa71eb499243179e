"""Paged caches for the GPU tests: seeded rows in shuffled pages, on the device and in float64."""
import numpy as np

from attention_fa2_forward_02_gb300 import synth
from oracle import serving as S
from tests import gpu_util as G


def codes_and_bytes(tag, shape):
    """Random finite e4m3 codes and scale bytes near 2^-6 .. 2^1."""
    raw = synth.counter_u16(tag + "/codes", shape)
    codes = (raw >> 8).astype(np.uint8)
    codes[(codes & 127) == 127] ^= 1
    exps = (121 + synth.counter_u16(tag + "/bytes", shape[:-1]) % 8).astype(np.uint8)
    return codes, exps


class Cache:
    """Pools of `spare` pages more than the sequences need, pages of `order` "hnd" or "nhd", filled from `tag`;
    `stale`: what lies in the slots past each length and in the spare pages ("nan", "inf" or None: more of the same)."""

    def __init__(self, tag, lens, page, hkv, d, dtype="bf16", e4m3=False, order="hnd", spare=2, stale=None, table_pages=None):
        import torch
        self.lens, self.page, self.hkv, self.d, self.dtype, self.e4m3 = list(lens), page, hkv, d, dtype, e4m3
        need = [-(-max(0, n) // page) for n in lens]
        self.pages = sum(need) + spare
        self.wide = table_pages or max(1, max(need))
        order_of = np.argsort(synth.raw_words(7, tag, 0, self.pages), kind="stable")
        self.table = np.full((len(lens), self.wide), -7, dtype=np.int32)  # entries past a length are not read
        at, used = 0, np.zeros((self.pages, page), dtype=bool)
        for b, n in enumerate(need):
            self.table[b, :n] = order_of[at:at + n]
            at += n
            for pos in range(lens[b]):
                used[self.table[b, pos // page], pos % page] = True
        shape = (self.pages, hkv, page, d)
        self.host, self.dev, self.exp = {}, {}, {}
        for side in "kv":
            if e4m3:
                codes, exps = codes_and_bytes(f"{tag}/{side}", shape)
                if stale:
                    codes[~np.broadcast_to(used[:, None], shape[:3])] = 0x7F
                self.host[side] = S.e4m3_values()[codes] * 2.0 ** (exps[..., None].astype(np.float64) - 127)
                t = torch.from_numpy(codes).cuda()
                self.exp[side] = torch.from_numpy(exps).cuda()
            else:
                x = synth.tensor(f"{tag}/{side}", shape, dtype)
                if stale:
                    bad = np.array([np.nan if stale == "nan" else np.inf])
                    x[~np.broadcast_to(used[:, None], shape[:3])] = synth.to_storage(bad, dtype)[0]
                self.host[side] = synth.widen(x, dtype)
                t = G.to_device(x, dtype)
            if order == "nhd":
                t = t.transpose(1, 2).contiguous().transpose(1, 2)
            self.dev[side] = t.view(torch.float8_e4m3fn) if e4m3 else t
        self.table_dev = torch.from_numpy(self.table).cuda()
        self.lens_dev = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def pools(self):
        return self.dev["k"], self.dev["v"]

    def exps(self):
        return {"k_exp": self.exp["k"], "v_exp": self.exp["v"]} if self.e4m3 else {}

    def rows(self, side, b):
        return S.rows_of(self.host[side], self.table[b], self.lens[b], self.page, self.pages)

    def value_exps(self, b, head):
        """The exponents of the value rows' scales (0 in a 16-bit cache), one for each token of sequence b."""
        length = min(max(int(self.lens[b]), 0), self.wide * self.page)
        out = np.zeros(length)
        if self.e4m3:
            exps = self.exp["v"].cpu().numpy()
            for pos in range(length):
                page = int(self.table[b, pos // self.page])
                out[pos] = int(exps[page, head, pos % self.page]) - 127 if 0 <= page < self.pages else 0
        return out
