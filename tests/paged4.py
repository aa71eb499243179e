"""Paged caches of 4-bit rows for the GPU tests, on the device and in float64."""
import numpy as np

from attention_fa2_forward_02_gb300 import synth
from oracle import serving as S
from tests.paged import Cache


class Cache4(Cache):
    """A Cache of 4-bit rows: random codes, scales of 2^-3 .. 30 and bytes near 2^-6 .. 2^1, so that every row's values have powers of two of
    their own; `stale`: NaN scales in the slots past each length and in the spare pages."""

    def __init__(self, tag, lens, page, hkv, d, dtype="bf16", order="hnd", stale=False, **kw):
        import torch
        super().__init__(tag, lens, page, hkv, d, dtype, True, order, **kw)
        shape = (self.pages, hkv, page)
        used = np.zeros((self.pages, page), dtype=bool)
        for b, n in enumerate(self.lens):
            for pos in range(n):
                used[self.table[b, pos // page], pos % page] = True
        self.scale, self.codes = {}, {}
        for side in "kv":
            codes = (synth.counter_u16(f"{tag}/{side}/codes4", shape + (d,)) >> 12).astype(np.uint8)
            scales = (32 + synth.counter_u16(f"{tag}/{side}/scales4", shape + (d // 16,)) % 64).astype(np.uint8)
            bytes_ = self.exp[side].cpu().numpy()
            if stale:
                scales[~np.broadcast_to(used[:, None], shape)] = 0x7F
            self.host[side] = S.row_values4(codes, scales, bytes_)
            t = torch.from_numpy(S.pack4(codes)).cuda()
            if order == "nhd":
                t = t.transpose(1, 2).contiguous().transpose(1, 2)
            self.dev[side] = t
            self.scale[side] = torch.from_numpy(scales).cuda().view(torch.float8_e4m3fn)
            self.codes[side] = codes

    def exps(self):
        return {"k_exp": self.exp["k"], "v_exp": self.exp["v"], "k_scale": self.scale["k"], "v_scale": self.scale["v"]}
