"""Oracle: rotary positions, the paged key-value cache and the attention of one new token, in float64.

Test infrastructure only.  Everything is written from the definitions in ``include/fa2.h``: rotations as
complex products, e4m3 codes by a search over the 256 values they stand for, the cache by walking tokens
one by one, the attention as an explicit softmax over the rows the block table names.

Inputs are float64 arrays (storage values already widened exactly).
"""
from __future__ import annotations

import numpy as np

MIN_EXP = -60


# ---------------------------------------------------------------------------- rotary positions
def rope(x, positions, inv_freq, interleaved, magnitude=1.0, backward=False):
    """x [B, H, N, d]; positions [B, N] integers; inv_freq [rot / 2]."""
    x = np.asarray(x, dtype=np.float64)
    r = len(inv_freq)
    angle = np.asarray(positions, dtype=np.float64)[:, None, :, None] * inv_freq
    turn = magnitude * np.exp((-1j if backward else 1j) * angle)
    one, two = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if interleaved else (slice(0, r), slice(r, 2 * r))
    z = (x[..., one] + 1j * x[..., two]) * turn
    y = x.copy()
    y[..., one], y[..., two] = z.real, z.imag
    return y


# ---------------------------------------------------------------------------- the 8-bit rows
def e4m3_values():
    """The values of codes 0 .. 255: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7f and 0xff are NaN."""
    out = np.empty(256)
    for code in range(256):
        sign, e, f = -1.0 if code & 128 else 1.0, (code >> 3) & 15, code & 7
        out[code] = np.nan if (code & 127) == 127 else sign * (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
    return out


def quantise_row(x):
    """(codes uint8 [d], scale byte) of one row."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.abs(x[np.isfinite(x)])
    a = finite.max() if finite.size else 0.0
    e = 0
    if a > 0:
        e = MIN_EXP
        while a > 448.0 * 2.0 ** e:
            e += 1
    y = x * 2.0 ** -e
    table = e4m3_values()[:127]  # codes 0 .. 126, ascending
    mag = np.minimum(np.abs(np.where(np.isnan(y), 0.0, y)), 448.0)
    dist = np.abs(table[None, :] - mag[:, None])
    low = dist.argmin(1)  # the lower of two codes at the same distance: adjacent ones
    tie = (low < 126) & (dist[np.arange(len(y)), np.minimum(low + 1, 126)] == dist[np.arange(len(y)), low])
    codes = np.where(tie & (low % 2 == 1), low + 1, low)  # ties: the even fraction
    codes = np.where(np.isnan(y), 0x7F, codes | np.where(np.signbit(y), 128, 0))
    return codes.astype(np.uint8), e + 127


def row_values(codes, byte):
    return e4m3_values()[codes] * 2.0 ** (int(byte) - 127)


# ---------------------------------------------------------------------------- the cache
def rows_of(pages, table, length, page_size, num_pages):
    """Rows [length, H, d] of one sequence out of pages [P, H, page_size, d], and which of them a page holds."""
    length = min(max(int(length), 0), len(table) * page_size)
    out = np.zeros((length, pages.shape[1], pages.shape[3]))
    held = np.zeros(length, dtype=bool)
    for pos in range(length):
        page = int(table[pos // page_size])
        if 0 <= page < num_pages:
            out[pos], held[pos] = pages[page, :, pos % page_size], True
    return out, held


def append_slots(table, lens, cu_new, page_size, num_pages):
    """[(row of k and v, page, slot)] of an append: cu_new None: one new token a sequence."""
    out = []
    for b, n in enumerate(lens):
        first, end = (b, b + 1) if cu_new is None else (int(cu_new[b]), int(cu_new[b + 1]))
        for t in range(first, end):
            pos = int(n) - end + t
            if not 0 <= pos < table.shape[1] * page_size:
                continue
            page = int(table[b][pos // page_size])
            if 0 <= page < num_pages:
                out.append((t, page, pos % page_size))
    return out


# ---------------------------------------------------------------------------- attention of one token
def decode_row(q, k, v, scale, live=None):
    """q [d], k, v [n, d] -> (o [d], lse, sum_j P_j |v_j| [d], max_j scale sum_d |q_d k_jd|); live [n]: the keys that count."""
    if live is not None:
        k, v = k[live], v[live]
    if len(k) == 0:
        return np.zeros(q.shape[0]), -np.inf, np.zeros(q.shape[0]), 0.0
    s = scale * (k @ q)
    m = s.max()
    p = np.exp(s - m)
    total = p.sum()
    return (p @ v) / total, m + np.log(total), (p @ np.abs(v)) / total, float(np.max(scale * (np.abs(k) @ np.abs(q))))
