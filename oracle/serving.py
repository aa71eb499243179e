"""Oracle: rotary positions, the paged key-value cache and the attention of one new token, in float64.

Test infrastructure only.  Everything is written from the definitions in ``include/fa2.h``: rotations as
complex products, e4m3 codes by a search over the 256 values they stand for, the cache by walking tokens
one by one, the attention as an explicit softmax over the rows the block table names.

Inputs are float64 arrays (storage values already widened exactly).
"""
from __future__ import annotations

import math

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


# ---------------------------------------------------------------------------- the 4-bit rows
E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _nearest_even(y, values):
    """Indices of the ascending `values` nearest to the magnitudes y, the even index of two at the same distance."""
    y = np.minimum(np.asarray(y, dtype=np.float64), values[-1])
    dist = np.abs(values[None, :] - y.reshape(-1, 1))
    low = dist.argmin(1)
    last = len(values) - 1
    tie = (low < last) & (dist[np.arange(len(low)), np.minimum(low + 1, last)] == dist[np.arange(len(low)), low])
    return np.where(tie & (low % 2 == 1), low + 1, low).reshape(np.shape(y))


def quantise_row4(x, before=None, more=0):
    """(codes 0 .. 15 [d], scale bytes [d / 16], byte) of one row.  `before`: the row before its rotation, whose power of
    two counts, raised by `more`."""
    x = np.asarray(x, dtype=np.float64)
    b = x if before is None else np.asarray(before, dtype=np.float64)
    finite = np.abs(b[np.isfinite(b)])
    a = finite.max() if finite.size else 0.0
    e = min((max(math.floor(math.log2(a)) - 9, MIN_EXP) if a > 0 else 0) + more, 120)
    y = (x * 2.0 ** -e).reshape(-1, 16)
    codes, scales = np.zeros(y.shape, dtype=np.uint8), np.zeros(len(y), dtype=np.uint8)
    e4m3 = e4m3_values()[:127]
    for g, row in enumerate(y):
        if np.isnan(row).any():
            scales[g] = 0x7F
            continue
        big = np.abs(row).max()
        scales[g] = 126 if np.isinf(big) else _nearest_even(np.array([big / 6]), e4m3)[0]
        s = e4m3[scales[g]]
        c = _nearest_even(np.abs(row) / s, E2M1_VALUES) if s > 0 else np.zeros(16, dtype=int)
        codes[g] = c | np.where(np.signbit(row), 8, 0)
    return codes.reshape(-1), scales, e + 127


def row_values4(codes, scales, byte):
    """What a 4-bit row stands for: codes 0 .. 15 [..., d], scale bytes [..., d / 16], bytes [...]."""
    codes = np.asarray(codes)
    v = E2M1_VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.repeat(e4m3_values()[np.asarray(scales)], 16, axis=-1)
    return v * s * 2.0 ** (np.asarray(byte, dtype=np.float64)[..., None] - 127)


def pack4(codes):
    """Two codes a byte, the even element in the low four bits."""
    c = np.asarray(codes, dtype=np.uint8)
    return c[..., ::2] | (c[..., 1::2] << 4)


# ---------------------------------------------------------------------------- bounds and selection
def smallest_exp(a, most):
    """The smallest e >= MIN_EXP with a <= most 2^e; 0 for a = 0."""
    if a == 0:
        return 0
    e = MIN_EXP
    while a > most * 2.0 ** e:
        e += 1
    return e


def page_bounds(keys):
    """(codes int [2, d], byte) of the live keys [n, d] of a page: lowest and highest of each channel, NaN not counted."""
    k = np.asarray(keys, dtype=np.float64)
    none = np.isnan(k).all(0)
    low = np.where(none, 0.0, np.min(np.where(np.isnan(k), np.inf, k), 0))
    high = np.where(none, 0.0, np.max(np.where(np.isnan(k), -np.inf, k), 0))
    finite = np.abs(k[np.isfinite(k)])
    e = smallest_exp(finite.max() if finite.size else 0.0, 127.0)
    return np.clip(np.stack([np.floor(low * 2.0 ** -e), np.ceil(high * 2.0 ** -e)]), -127, 127).astype(np.int64), e + 127


def touched_pages(lens, cu_new, page_size, room):
    """{(sequence, page number in it): live keys} of the pages that new tokens lie in."""
    out = {}
    for b, n in enumerate(lens):
        count = 1 if cu_new is None else int(cu_new[b + 1]) - int(cu_new[b])
        end = min(max(int(n), 0), room)
        for pos in range(max(0, int(n) - count), end):
            out[b, pos // page_size] = min(page_size, end - pos // page_size * page_size)
    return out


def query_integers(q):
    """(integers [d], e) of one query row."""
    q = np.where(np.isnan(q), 0.0, np.asarray(q, dtype=np.float64))
    finite = np.abs(q[np.isfinite(q)])
    e = smallest_exp(finite.max() if finite.size else 0.0, 127.0)
    return np.clip(np.rint(q * 2.0 ** -e), -127, 127).astype(np.int64), e


def page_score(qs, codes, byte):
    """The score of a page with bounds codes [2, d] for the query rows qs [group, d]."""
    best = -math.inf
    for q in qs:
        ints, e = query_integers(q)
        best = max(best, int(np.maximum(ints * codes[0], ints * codes[1]).sum()) * 2.0 ** e)
    return best * 2.0 ** (int(byte) - 127)


def select_pages(scores, budget, first, recent):
    """The numbers of the pages taken, ascending; scores: None for a page outside the cache."""
    n = len(scores)
    rank = lambda j: (0 if j < first or j >= n - recent else 1 if scores[j] is not None else 2,  # noqa: E731
                      -scores[j] if 0 <= j < n and scores[j] is not None and not (j < first or j >= n - recent) else 0.0, j)
    return sorted(sorted(range(n), key=rank)[:budget])
