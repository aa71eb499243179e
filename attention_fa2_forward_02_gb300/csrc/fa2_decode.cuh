// fa2_decode.cuh - attention of one new token of each sequence over a paged key-value cache.
//
// fa2_forward's formula for one query row a head: O = softmax(scale q K^T) V, LSE, over the
// sequence's cached keys. Every key and value is read once for up to 16 query heads, 4 * 16
// FLOPs for 4 bytes at most, so memory sets the pace and the products only have to keep up:
// they run as warp-level 16 x 8 x 16 products on registers. Their 16 rows are keys in the
// first (S^T = K Q^T) and columns of V in the second (O^T = V^T P^T), their 8 columns query
// heads of one key-value head: K and V come out of shared memory as whole left operands, and
// up to 8 heads cost no more than one. (The 128-row products of the tensor memory path would
// want the probabilities back through shared memory for every tile.)
//
// Work: the keys of every (sequence, key-value head, 8 or 16 query heads) item are cut into blocks
// of kKeys; all blocks of all items in a row are divided evenly over the CTAs, whatever the
// lengths, and a CTA's blocks of one item over its warps, one by one. Each warp keeps its own
// running maximum, sum and O, and its own ring of stages filled by asynchronous 16-byte copies
// that run ahead of the products, over the ends of items too: while the CTA adds its warps'
// results up in shared memory at the end of an item, the copies for the next one are under way.
// An item that lies in one CTA is then done, the others leave (m, l, O) in the workspace, at
// most two per CTA, and the second kernel joins them in CTA order. An item counts as kOver
// blocks more than it has, the time its end takes: else the CTA that gets a short sequence's
// many heads finishes last.
//
// The 8-bit cache: with key scale 2^a and value scale 2^e per row, the score of a key is
// s = scale log2(e) 2^a (q . codes), its weight P = 2^(x - m) with x = s + e and m a maximum of x:
// the value's scale is inside the weight, and the second product runs on bare codes. The
// denominator has a maximum ml of its own, l = sum 2^(s - ml): scales lie up to 2^180 apart, and
// counted as P 2^-e a key of small values would be gone from the sum before 2^-e could bring it
// back. O = sum P codes / l * 2^(m - ml). Rows of zeros are stored with e = 0, often far above the
// others' and next to nothing in O: they do not raise m. Codes are exact in half; q (bfloat16) is
// brought to half exactly by a power of two of its row's largest element.
//
// The 4-bit cache is the same with code * scale, 6 bits and exact in half, in the place of the code: K's and V's
// operands are made in registers (a byte of two codes to a pair of halves, times the group's scale; the lanes' pieces
// of a row are permuted alike on both sides of a product, so no element moves between lanes). Not its 73 bytes a row bound
// it but the chain of a block: conversion, product, maximum, exponential, second product, 420 instructions for 16 keys of 128
// by three warps a scheduler, issued in 58 of 100 cycles; no unit is busy for more than 47. GB300, 32
// sequences of up to 8192 (d 128, 8 heads on each of 8, 193 MB): 56 us, 3.5 TB/s; 21 of up to 65536 (d 64, half, 507
// MB): 159 to 168 us, 3.0 to 3.2 TB/s, where each weight takes two products.
//
// Contexts that can only be short (by the block table's width, or the window) take one launch: the
// CTAs of a thread-block cluster share an item and join their results in distributed shared
// memory. GB300, one sequence of 1000 tokens, 8 heads: 8.5 us in two launches, 6.7 in one.
#pragma once

#include <algorithm>

#include "paged.cuh"

namespace fa2 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kOver = 8;          // blocks an item counts beyond its own
constexpr int kJoinThreads = 512;
constexpr int kFewItems = 4;      // items up to which (twice which) it joins one row (two) per CTA
constexpr float kRescale = 8.0f;  // the running maximum may lag by this much (base-2 units) before O is rescaled
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kNoScore = -3.402823466e38f;  // a maximum of no scores, from which -infinity can be subtracted

// D: the head size's kernel; kForm: the cache's type (CacheForm); kTiles: query heads per item / 8.
template <int D, int kForm, int kTiles>
struct Cfg {
    static constexpr bool kCodes = kForm != kRows16, kE4m3 = kForm == kRowsE4m3, kE2m1 = kForm >= kRowsE2m1;
    static constexpr bool kSixteens = kForm == kRowsE2m1By16;  // (DecodeParams::by_sixteens)
    static constexpr int kRowBytes = kE2m1 ? D / 2 : (kE4m3 ? D : 2 * D);
    static constexpr int kRows = 8 * kTiles;                // query heads per item
    // CTAs an SM. 16-bit rows keep memory busy with two, and three read unevenly fast (21 sequences of
    // up to 65536, 8 heads: d 128 567 -> 634 us, d 64 317 -> 341). e4m3 has more to do per byte: 32
    // sequences of up to 8192, a one-token one among them, d 128 76 us with two and 65 with three (long
    // contexts 304 and 322), d 32 34 and 33. But three leave 168 registers: too few at d 64, 8 heads
    // (41 us with two, 50 with three; long 163 and 198), and for 16 heads (d 64 57 and 70, d 128 86
    // and 155; d 32 42 and 40). 4-bit rows have the most to do: batch of 32, d 128, 75 us with two and 70 with three
    // (four spill: 76).
    static constexpr int kPerSm = (kE4m3 && (D == 32 || (D == 128 && kTiles == 1))) || (kE2m1 && kTiles == 1) ? 3 : 2;
    static constexpr int kMaxCtas = 152 * kPerSm;           // a fixed number: the split depends on the lengths alone
    // in one launch, where latency is more than memory: 7 windows of 1024 keys, d 64, 9.6 -> 8.8 us
    static constexpr int kShortPerSm = kTiles == 1 && kRowBytes < 256 ? 3 : kPerSm;
    // keys per block: 8 KB of K and V (4 of 32-byte rows, and of 4-bit rows at d 128)
    static constexpr int kKeys = kRowBytes >= 256 ? 16 : (kRowBytes == 128 || (kE2m1 && D == 128) ? 32 : 64);
    static constexpr int kLooks = (kKeys + 31) / 32;        // keys a lane looks up per block
    static constexpr int kChunks = kRowBytes / 16;          // 16-byte chunks a row
    static constexpr int kTile = kKeys * kRowBytes;         // K or V of a block
    // Rows that are no whole lines of 128 bytes are fetched by halves of lines: left to itself L2
    // fetches the other half of a row's last line too, which in a token-major cache is another
    // head's row and gone again before that head's CTA comes to it. Token-major, 8 heads, 21
    // sequences of up to 65536 tokens in 16 bits: d 96 531 -> 466 us, d 48 420 -> 359, d 32 256 ->
    // 172; 32 of up to 8192 in e4m3: d 64 50 -> 40, d 96 82 -> 74. Whole lines of 16-bit rows were
    // 1% slower by halves, so there d is asked; those of e4m3 rows were not.
    static constexpr bool kHalfLines = kCodes || kRowBytes <= 64;
    static constexpr int kInfo = kCodes ? kKeys * 8 : 16;   // codes: a float2 per key; else the keys that count, as bits
    static constexpr int kScaleRow = D / 16;                // e2m1: scale bytes of a key
    static constexpr int kScales = kE2m1 ? kKeys * kScaleRow : 0;  // and of a block's keys, or values
    static constexpr int kExps = 2 * kTile + kInfo + 2 * kScales;  // e2m1: bytes of K's, then V's powers of two
    static constexpr int kStage = kExps + (kE2m1 ? 2 * kKeys : 0);
    // 4-bit rows at d 128: a block of 4.7 KB is too little on its way a warp. Batch of 32 69.6 us with two stages, 65.0
    // with three (and keys looked up by teams of lanes, below); d 64, whose blocks hold 64 keys: no gain from three or four.
    static constexpr int kStages = kE2m1 && D == 128 ? 3 : 2;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kQ = kRows * D * 2;                // q as the first product takes it
    static constexpr int kPitch = kCodes ? D + 8 : D + 4;    // floats a row at the end of an item (no bank twice)
    static constexpr int smem(int merge_rows) { return kRing + kQ + kWarps * merge_rows * kPitch * 4 + kRows * 4; }
    static constexpr bool fits(int bytes) { return bytes + 1024 + 256 <= 228 * 1024 / kShortPerSm; }
    // rows the warps add up at a time there: as many as find room
    static constexpr int kMergeRows = fits(smem(8)) ? 8 : (fits(smem(4)) ? 4 : 2);
    static constexpr int kMerge = kWarps * kMergeRows * kPitch * 4;
    static constexpr int kSmem = smem(kMergeRows);
    static_assert(fits(kSmem), "CTAs an SM");
};

// Position of chunk `c` of row `r` in a tile: the eight rows an ldmatrix reads at one chunk lie
// in eight different 16-byte bank groups.
template <int kChunks>
__device__ __forceinline__ int swizzle(int r, int c) {
    if constexpr (kChunks >= 8) return r * kChunks + (c ^ (r & 7));
    else if constexpr (kChunks == 4) return r * 4 + (c ^ ((r >> 1) & 3));
    else if constexpr (kChunks == 2) return r * 2 + (c ^ ((r >> 2) & 1));
    else return r;
}

// bytes: 16, or 0 (nothing is read, the 16 bytes are filled with zeros)
// Always or half: L2 fetches 64 bytes for this and no more
template <bool kAlways>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes, bool half) {
    if (kAlways || half)
        asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// kBytes: 4 or 8, read where `on`, else zeros
template <int kBytes>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(on ? kBytes : 0) : "memory");
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((uint16_t)v) : "memory");
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory"); }
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// 4-bit rows. Which 16 keys and which of their codes are a product's rows and terms is free, as long as the other operand has
// the same order, so each lane takes codes that lie together: for the scores, of a key, the D / 4 from D / 4 t on (a piece of
// 16, 8 or 4 bytes, one or two scales), for O, of four keys, the D / 8 from D / 8 g on (8, 4 or 2 bytes, a scale a key).
// Row r of eight is key key_of(r), an order in which neither reads a bank twice: D = 128 0 3 4 7 1 2 5 6, 64 0 6 1 7 2 4 3 5.
// (As matrix loads bring them, with 4 scales a key and side and pairs of keys made after the conversion: batch of 32 57.3 us,
// 55.8 so; in half 62.7 and 59.5; 21 contexts of up to 65536 at d 128 257 and 242; d 32 27.6 and 28.2.)
template <int D>
__device__ __forceinline__ int key_of(int r) {
    return D == 128 ? (0x65217430u >> (4 * r)) & 7 : (D == 64 ? (0x53427160u >> (4 * r)) & 7 : r);
}

// A key's scales for each 8 of this lane's codes, as pairs of the same half; `row`: the key's D / 16 bytes.
template <int D>
__device__ __forceinline__ void key_scales(uint32_t row, int t, uint32_t (&s)[D / 32]) {
    if constexpr (D == 128) {
        const uint32_t two = e4m3x2_to_f16x2(ld_shared_u16(row + 2 * t));
        s[0] = s[1] = __byte_perm(two, 0, 0x1010);
        s[2] = s[3] = __byte_perm(two, 0, 0x3232);
    } else {
        const uint32_t one = e4m3x2_to_f16x2(ld_shared_u8(row + (D == 64 ? t : t / 2)) * 0x101u);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) s[i] = one;
    }
}

// A lane's codes of a key: D / 8 bytes (kHalf: D / 16), in words.
template <int D, bool kHalf>
__device__ __forceinline__ void lane_codes(uint32_t addr, uint32_t (&w)[kHalf ? (D + 63) / 64 : D / 32]) {
    constexpr int kBytes = kHalf ? D / 16 : D / 8;
    if constexpr (kBytes == 16) {
        const uint4 x = ld_shared_v4(addr);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else if constexpr (kBytes == 8) {
        const uint2 x = ld_shared_v2(addr);
        w[0] = x.x, w[1] = x.y;
    } else if constexpr (kBytes == 4) {
        w[0] = ld_shared_u32(addr);
    } else {
        w[0] = ld_shared_u16(addr);
    }
}

// The transpose of an 8 x 8 matrix of 16-bit elements, row g, columns 2t, 2t+1 in lane 4 g + t.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kBf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// a / b for a >= 0, b > 0: the 32-bit division where both fit (the 64-bit one is far longer).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// How the units (units_of) of all items are divided over the CTAs: evenly, the first `rest` CTAs
// one more. Items are ordered by (sequence, head block); every sequence has `per_seq` of them,
// with the same number of blocks.
struct Split {
    int64_t share, rest;
    int ctas;  // CTAs that have any: at least a unit for each of their warps
    __device__ __forceinline__ Split(int64_t total, int max_ctas) {
        const int64_t n = (total + kWarps - 1) / kWarps;
        ctas = n < max_ctas ? (int)n : max_ctas;
        share = ctas ? quotient(total, ctas) : 0;
        rest = total - share * ctas;
    }
    __device__ __forceinline__ int64_t begin(int64_t c) const { return c * share + (c < rest ? c : rest); }
    // the CTA that unit u belongs to
    __device__ __forceinline__ int owner(int64_t u) const {
        const int64_t longer = rest * (share + 1);
        const int64_t c = u < longer ? quotient(u, share + 1) : rest + quotient(u - longer, share);
        return c < ctas ? (int)c : ctas - 1;
    }
};

// The keys [first, len) of sequence b that the window leaves; its blocks begin at `base`, a
// multiple of 16, so that 16 keys lie in one page where the page size is one too.
struct Range {
    int base, first, len;
};
__device__ __forceinline__ Range range_of(const DecodeParams& p, int b) {
    const int len = bounded_len(p.c.lens[b], p.c.room, p.c.status);
    const int first = p.window > 0 && len > p.window ? (int)(len - p.window) : 0;
    return {first & ~15, first, len};
}
template <int kKeys>
__device__ __forceinline__ int blocks_of(Range r) { return (r.len - r.base + kKeys - 1) / kKeys; }
// What an item of `nb` blocks counts in the division of the work.
__device__ __forceinline__ int units_of(int nb) { return nb ? nb + kOver : 0; }

// What a share of a row's keys leaves beside its O (relative to 2^m): l relative to 2^ml.
// (16-bit caches: ml = m.)
struct __align__(16) Stats {
    float m, l, ml, unused;
};

// The factors that bring the O and l of a share to the larger references (m, ml).
template <bool kCodes>
struct Factors {
    float o, l;
    __device__ __forceinline__ Factors(const Stats& s, float m, float ml) {
        o = ex2_approx(s.m - (m == -INFINITY ? 0.f : m));
        l = kCodes ? ex2_approx(s.ml - ml) : o;
    }
};

// A row's last step: O = sum P V times scale(), LSE.
template <bool kCodes>
struct Last {
    float inv, half, lse;
    __device__ __forceinline__ Last(float m, float ml, float l) {
        inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        half = kCodes ? ex2_approx(0.5f * (m - ml)) : 1.f;  // twice: m - ml reaches 120 and more
        lse = l == 0.f ? -INFINITY : ((kCodes ? ml : m) + lg2_approx(l)) * kLn2;
    }
    __device__ __forceinline__ float operator()(float a) const { return kCodes ? a * half * inv * half : a * inv; }
};

// Workspace: per CTA two partial results (its first item, if that began before it or ends after
// it; its last item, if that ends after it), each [kRows][D] floats and then [kRows] Stats;
// behind all of them, per CTA, the item that begins in it and ends in a later CTA. (The second
// kernel could find that from the lengths, but while the first one fills the SMs it has no place
// to do so early: 3 us of the e4m3 batch.)
template <int D, int kRows>
__device__ __forceinline__ float* partial(float* ws, int64_t cta, int which) {
    return ws + (cta * 2 + which) * (kRows * (D + 4));
}

struct __align__(16) Torn {
    int rows;      // 0: none
    int last_cta;
    int which;     // the first CTA's partial result
    int out_row;   // row of O and LSE
};
template <typename C, int D>
__device__ __forceinline__ Torn* torn(float* ws, int64_t cta) {
    return reinterpret_cast<Torn*>(partial<D, C::kRows>(ws, C::kMaxCtas, 0)) + cta;
}

// A place in the order of items: sequence b, whose first unit is u_seq.
struct Place {
    int64_t u_seq;
    Range range;
    int b;
};
struct LocateSmem {
    int64_t sums[kWarps];
    Place place;
};

// Inclusive sums over the CTA's threads in order, and the total of all.
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t* sums, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sums[w];
        all += sums[w];
    }
    *total = all;
    return before + v;
}

// The division of all sequences' units over the CTAs, CTA blockIdx.x's share [u_begin, u_end) of
// them, and the place of its first unit. All threads call it; false: the CTA has no share, and no
// place.
template <int kKeys>
__device__ __forceinline__ bool locate(const DecodeParams& p, int64_t per_seq, int max_ctas, LocateSmem& sm, Split* split,
                                       int64_t* u_begin, int64_t* u_end) {
    const int batch = (int)p.c.batch, per = (batch + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, batch), b1 = min(b0 + per, batch);  // this thread's sequences
    int64_t mine = 0, total;
    Range range{0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        range = range_of(p, b);
        mine += units_of(blocks_of<kKeys>(range));
    }
    int64_t upto = cta_scan(mine, sm.sums, &total);
    *split = Split(total * per_seq, max_ctas);
    if ((int)blockIdx.x >= split->ctas) return false;
    *u_begin = split->begin(blockIdx.x);
    *u_end = split->begin(blockIdx.x + 1);
    upto -= mine;
    if (upto * per_seq <= *u_begin && *u_begin < (upto + mine) * per_seq) {  // among this thread's sequences
        int b = b0;
        if (per > 1)
            for (;; ++b) {
                range = range_of(p, b);
                const int units = units_of(blocks_of<kKeys>(range));
                if (*u_begin < (upto + units) * per_seq || b + 1 >= b1) break;  // (b1: lengths written meanwhile)
                upto += units;
            }
        sm.place = Place{upto * per_seq, range, b};
    }
    __syncthreads();
    return true;
}

template <bool kBf16>
__device__ __forceinline__ void put(void* o, int64_t i, float v) {
    if constexpr (kBf16) static_cast<__nv_bfloat16*>(o)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(o)[i] = __float2half_rn(v);
}

// A CTA's blocks [k0, k1) of one item, and where the item lies.
struct Segment {
    int64_t u_seq;  // first unit of sequence b
    int64_t next;   // first unit behind the item
    Range range;    // of sequence b
    int b, nb;      // its blocks
    int item, k0, k1;
};

// Joins the shares [kRows][D], [kRows] Stats that each CTA of the cluster has at `part` in its
// shared memory, in rank order: CTA r writes rows r, r + ranks, ... Every thread of the cluster calls it.
template <int D, bool kBf16, bool kCodes, int kRows>
__device__ __forceinline__ void join_cluster(const DecodeParams& p, uint32_t part, int ranks, int rank, int rows, int64_t out_row) {
    cluster_sync_all();
    const int d = threadIdx.x;  // D <= kThreads: a column a thread
    for (int r = rank; r < rows; r += ranks) {
        if (d >= D) continue;
        auto stats = [&](int k) {
            const uint32_t at = cluster_map(part + (kRows * D + 4 * r) * 4, k);
            Stats s;
            s.m = ld_cluster(at);
            s.l = ld_cluster(at + 4);
            s.ml = kCodes ? ld_cluster(at + 8) : s.m;
            return s;
        };
        float m = -INFINITY, ml = -INFINITY, a = 0.f, l = 0.f;
        for (int k = 0; k < ranks; ++k) {
            const Stats s = stats(k);
            m = fmaxf(m, s.m);
            ml = fmaxf(ml, s.ml);
        }
        for (int k = 0; k < ranks; ++k) {
            const Stats s = stats(k);
            const Factors<kCodes> f(s, m, ml);
            l += f.l * s.l;
            a += f.o * ld_cluster(cluster_map(part + (r * D + d) * 4, k));
        }
        const Last<kCodes> last(m, ml, l);
        if (d < p.c.d) put<kBf16>(p.o, (out_row + r) * p.c.d + d, last(a));
        if (d == 0) p.lse[out_row + r] = last.lse;
    }
    cluster_sync_all();  // no CTA leaves while another reads its shared memory
}

// kPerHead: block table and lengths for each (sequence, key-value head) pair, which then counts as a sequence.
// kCluster: the CTAs of a cluster of `ranks` share the item blockIdx.x / ranks; nothing is left to
// the second kernel.
template <int D, bool kBf16, int kForm, int kTiles, bool kPerHead, bool kCluster>
__global__ void __launch_bounds__(kThreads, kCluster ? Cfg<D, kForm, kTiles>::kShortPerSm : Cfg<D, kForm, kTiles>::kPerSm)
    fa2_decode_kernel(const DecodeParams p, int ranks) {
    using C = Cfg<D, kForm, kTiles>;
    constexpr bool kCodes = C::kCodes, kE4m3 = C::kE4m3, kE2m1 = C::kE2m1;
    constexpr bool kMmaBf16 = kBf16 && !kCodes;
    // m lies this much below the maximum it was taken from: weights 2^-(14 + kLift) of the largest
    // still have all of half's bits (bfloat16 has float32's exponents)
    constexpr float kLift = kMmaBf16 ? 0.f : 7.f;
    // Whether the product with V takes what a weight's rounding to 16 bits left off as well: it is the
    // largest error of O but where a half weight's 2^-11 stands beside a bfloat16 result's 2^-8. (e4m3
    // with bfloat16, batch of 32: 8 heads 66.0 us in one product and 67.7 in two, 16 heads 79.8 and
    // 85.5; 16-bit long contexts, bound by memory, the same.)
    constexpr bool kRest = !(kCodes && kBf16);
    constexpr int kKeys = C::kKeys, S = C::kStages, kRows = C::kRows, kMt = kKeys / 16, kMR = C::kMergeRows;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LocateSmem located;
    const PagedParams& c = p.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = p.heads / c.hkv, hblocks = (group + kRows - 1) / kRows;
    const int64_t per_seq = kPerHead ? hblocks : (int64_t)c.hkv * hblocks;
    grid_begin();

    Split split(0, 0);
    int64_t u_begin = 0, u_end = 0;
    // rows without a key, strewn over the CTAs
    auto empty_rows = [&]() {
        for (int b = blockIdx.x; b < c.batch; b += gridDim.x) {
            if (range_of(p, b).len > 0) continue;
            const int rows = kPerHead ? group : p.heads;
            const int64_t row0 = (int64_t)b * rows;
            for (int i = threadIdx.x; i < rows * c.d / 8; i += kThreads)
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row0 * c.d)[i] = make_uint4(0, 0, 0, 0);
            for (int i = threadIdx.x; i < rows; i += kThreads) p.lse[row0 + i] = -INFINITY;
        }
    };
    if constexpr (!kCluster) {
        if (!locate<kKeys>(p, per_seq, gridDim.x, located, &split, &u_begin, &u_end)) {
            if (threadIdx.x == 0) torn<C, D>(p.workspace, blockIdx.x)->rows = 0;
            empty_rows();
            return;
        }
    }

    // the segment that unit u lies in; false: the CTA has no block from u on
    auto seek = [&](Segment& s, int64_t u) {
        if constexpr (kCluster) {
            return false;  // there is but one
        } else {
            if (u >= u_end) return false;
            while (u >= s.u_seq + units_of(s.nb) * per_seq) {
                if (s.b + 1 >= c.batch) return false;  // (only with lengths written meanwhile)
                s.u_seq += units_of(s.nb) * per_seq;
                s.range = range_of(p, ++s.b);
                s.nb = blocks_of<kKeys>(s.range);
            }
            const int units = units_of(s.nb);
            if (units == 0) return false;  // (the same)
            s.item = (int)quotient(u - s.u_seq, units);
            const int64_t u_item = s.u_seq + (int64_t)s.item * units;  // kOver units first, then the blocks
            const int64_t from = u - u_item - kOver, to = u_end - u_item - kOver;
            s.k0 = from > 0 ? (int)from : 0;
            s.k1 = to < s.nb ? (int)to : s.nb;
            s.next = u_item + units;
            return s.k1 > s.k0;
        }
    };
    // this warp's blocks of segment number `number`: k0 + turn(number), + kWarps, ...
    auto turn = [&](int number) { return (warp + number) % kWarps; };
    auto count = [&](const Segment& s, int number) {
        const int n = s.k1 - s.k0 - turn(number);
        return n > 0 ? (n + kWarps - 1) / kWarps : 0;
    };

    Segment seg;
    bool live = true;
    const int rank = kCluster ? (int)blockIdx.x % ranks : 0;
    if constexpr (kCluster) {  // a share of the item, perhaps an empty one
        const int64_t number = blockIdx.x / ranks;
        seg.b = (int)quotient(number, per_seq);
        seg.item = (int)(number - seg.b * per_seq);
        seg.range = range_of(p, seg.b);
        seg.nb = blocks_of<kKeys>(seg.range);
        seg.k0 = (int)((int64_t)seg.nb * rank / ranks);
        seg.k1 = (int)((int64_t)seg.nb * (rank + 1) / ranks);
        seg.u_seq = seg.next = 0;
    } else {
        seg.b = located.place.b;
        seg.u_seq = located.place.u_seq;
        seg.range = located.place.range;
        seg.nb = blocks_of<kKeys>(seg.range);
        live = seek(seg, u_begin);
    }

    // ---- the ring. Lane r looks keys r, r + 32 of a block up; the page numbers are read one block
    // ahead of the copies (`ahead`), the scale bytes with the copies and stored one block later.
    uint8_t* my = smem + warp * S * C::kStage;
    const uint32_t my_addr = smem_u32(my);
    Segment ahead = seg;
    bool ahead_live = live;
    int ahead_number = 0, ahead_left = 0, ahead_key = 0;  // blocks of this warp left, the next one's first key
    const int32_t* ahead_table = nullptr;
    int64_t ahead_head = 0, ahead_exp = 0;                // the head's offset in a page, in its scale bytes
    uint32_t ahead_head16 = 0, ahead_head_key = 0;        // (by sixteens)
    auto enter = [&]() {
        if (!ahead_live) return;
        const int hk = kPerHead ? ahead.b % c.hkv : ahead.item / hblocks;
        ahead_left = count(ahead, ahead_number);
        ahead_key = ahead.range.base + (ahead.k0 + turn(ahead_number)) * kKeys + (kE2m1 ? 0 : (kKeys < 32 ? lane % kKeys : lane));
        ahead_table = c.table + ahead.b * c.table_stride;
        ahead_head = hk * c.head_stride;
        ahead_exp = (int64_t)hk * c.page_size;
        ahead_head16 = (uint32_t)hk * (uint32_t)(c.head_stride >> 4);
        ahead_head_key = (uint32_t)(hk * c.page_size);
    };
    enter();
    // e2m1, and pages of whole sixteens of keys: kTeam lanes look 16 keys of a block up, which lie after one another in
    // a page, and copy them: no address crosses lanes. (One key a lane, as below, took 390 instructions a block of 32
    // keys, more than its products.)
    const bool sixteens = c.page_size % 16 == 0;
    const bool by_sixteens = C::kSixteens;
    constexpr int kTeam = kE2m1 ? 512 / kKeys : 32;
    int page[C::kLooks], slot[C::kLooks];  // slot -1: no such key
    int64_t head_off = 0, head_exp = 0;    // and the block's head
    uint32_t head16 = 0, head_key = 0;     // (by sixteens)
    bool found = false;
    auto look = [&]() {  // the next block of this warp, if there is one
        while (ahead_live && ahead_left == 0) {
            ahead_live = seek(ahead, ahead.next);
            ++ahead_number;
            enter();
        }
        found = ahead_live;
        if (!found) return;
        head_off = ahead_head;
        head_exp = ahead_exp;
        if (by_sixteens) {
            head16 = ahead_head16;
            head_key = ahead_head_key;
            const int key = ahead_key + 16 * (lane / kTeam);
            page[0] = 0;
            slot[0] = -1;
            if (key + 15 >= ahead.range.first && key < ahead.range.len) {
                const int at = page_of(c, key);
                page[0] = ahead_table[at];
                slot[0] = key - at * c.page_size;
            }
            ahead_key += kWarps * kKeys;
            --ahead_left;
            return;
        }
#pragma unroll
        for (int j = 0; j < C::kLooks; ++j) {
            const int key = ahead_key + (kE2m1 ? lane : 0) + 32 * j;
            page[j] = 0;
            slot[j] = -1;
            if (key >= ahead.range.first && key < ahead.range.len) {
                const int at = page_of(c, key);
                page[j] = ahead_table[at];
                slot[j] = key - at * c.page_size;
            }
        }
        ahead_key += kWarps * kKeys;
        --ahead_left;
    };
    // a lane copies chunk lane % kChunks of every kStep-th row; past the head's size it fills with zeros
    const int lane_bytes = lane % C::kChunks * 16 < (kE2m1 ? c.d / 2 : (kE4m3 ? c.d : 2 * c.d)) ? 16 : 0;
    const int64_t lane_off = lane / C::kChunks * c.slot_stride + (lane_bytes ? lane % C::kChunks * 16 : 0);
    const int64_t rows_off = 32 / C::kChunks * c.slot_stride;
    const bool half_lines = c.d * 2 % 128 != 0;
    int fill = 0;                        // the stage to fill next
    uint32_t ka[C::kLooks], ve[C::kLooks];  // scale bytes of the block loaded last; ve 256: the key does not count
    int info_stage = -1;                 // and its stage, while they are not stored
    // e2m1, key by key: the scale bytes of the keys `some` at `at` into K's and V's scales at `dst`
    auto load_scales = [&](uint32_t dst, const uint32_t (&some)[C::kLooks], const int64_t (&at)[C::kLooks]) {
        if constexpr (kE2m1) {
            const int row = c.d / 16;  // bytes a key has in memory
#pragma unroll
            for (int j = 0; j < C::kLooks; ++j) {
                const bool on = (some[j] >> lane) & 1u;
                const uint8_t *ks = c.k_scale + (on ? at[j] * row : 0), *vs = c.v_scale + (on ? at[j] * row : 0);
                const uint32_t to = dst + (lane + 32 * j) * C::kScaleRow;
                if (D >= 64 && row == C::kScaleRow) {
                    cp_async_small<C::kScaleRow>(to, ks, on);
                    cp_async_small<C::kScaleRow>(to + C::kScales, vs, on);
                } else {  // rows of 2 or 6 bytes have no asynchronous copy
                    for (int e = 0; e < C::kScaleRow; e += 2) {
                        st_shared_u16(to + e, on && e < row ? *reinterpret_cast<const uint16_t*>(ks + e) : 0);
                        st_shared_u16(to + C::kScales + e, on && e < row ? *reinterpret_cast<const uint16_t*>(vs + e) : 0);
                    }
                }
            }
        }
    };
    // e2m1, by sixteens: this lane's pieces of its team's 16 keys. A team's rows are copied whole if any of them counts (a
    // page holds all 16), and not at all otherwise: a code that does not count is finite whatever it is. Scales are not,
    // and become zeros (here where none counts, else in tidy_scales).
    const int team = lane / kTeam, mate = lane % kTeam, mate_row = mate / C::kChunks, mate_piece = mate % C::kChunks;
    constexpr int kTeamRows = kTeam / C::kChunks;  // rows a copy covers
    const uint32_t step16 = (uint32_t)(c.slot_stride >> 4), mate16 = mate_row * step16 + mate_piece;
    const bool mate_on = 32 * mate_piece < c.d;
    // scale bytes: 16 keys' are d contiguous ones, D / 16 pieces of K and as many of V (d = 96: rows of 6 bytes, widened
    // later); after those, for the powers of two, a piece of K and a piece of V
    constexpr int kPer = D / 16;
    const int scale_side = mate / kPer, scale_piece = mate % kPer;
    const bool scale_on = scale_side < 2 && 16 * scale_piece < c.d;
    auto load_sixteens = [&](uint32_t st) {
        if constexpr (kE2m1) {
            const bool there = slot[0] >= 0 && (uint32_t)page[0] < (uint64_t)c.num_pages;
            if (slot[0] >= 0 && !there && c.status) atomicOr(c.status, kStatusBadIndex);
            // in units of 16 bytes, and of keys: within 32 bits (by_sixteens)
            const uint32_t o = there ? (uint32_t)page[0] * (uint32_t)(c.page_stride >> 4) + (uint32_t)slot[0] * step16 + head16 + mate16 : 0u;
            const uint32_t e = there ? (uint32_t)page[0] * (uint32_t)(c.hkv * c.page_size) + (uint32_t)slot[0] + head_key : 0u;
            if (there && mate_on) {
                const char *ks = c.k + (uint64_t)o * 16, *vs = c.v + (uint64_t)o * 16;
#pragma unroll
                for (int i = 0; i < 16 / kTeamRows; ++i) {
                    const uint32_t dst = st + swizzle<C::kChunks>(16 * team + i * kTeamRows + mate_row, mate_piece) * 16;
                    cp_async16<true>(dst, ks, 16, true);
                    cp_async16<true>(dst + C::kTile, vs, 16, true);
                    ks += kTeamRows * c.slot_stride;
                    vs += kTeamRows * c.slot_stride;
                }
            }
            const int bytes = there ? 16 : 0;  // else zeros
            if (scale_on)
                cp_async16<true>(st + 2 * C::kTile + C::kInfo + scale_side * C::kScales + 16 * team * C::kScaleRow + scale_piece * 16,
                                 (scale_side ? c.v_scale : c.k_scale) + ((uint64_t)e * (uint32_t)(c.d / 16) + (there ? scale_piece * 16 : 0)), bytes, true);
            if (mate < 2) cp_async16<true>(st + C::kExps + mate * kKeys + 16 * team, (mate ? c.v_exp : c.k_exp) + e, bytes, true);
        }
    };
    auto load = [&]() {  // copies the block looked up last into the next stage; commits one group
        if (found && by_sixteens) {
            load_sixteens(my_addr + fill * C::kStage);
        } else if (found) {
            const uint32_t st = my_addr + fill * C::kStage;
            const char* kbase = c.k + head_off;
            const char* vbase = c.v + head_off;
            int64_t off[C::kLooks];
            uint32_t some[C::kLooks];  // the keys that count, as bits
            int64_t scale_at[C::kLooks];  // e2m1: the key's place among the scale bytes
#pragma unroll
            for (int j = 0; j < C::kLooks; ++j) {
                Slot s{-1, -1};
                if (slot[j] >= 0) s = slot_of(c, page[j], slot[j]);
                off[j] = s.off;
                some[j] = __ballot_sync(0xffffffffu, s.off >= 0);
                if constexpr (kCodes) {
                    const int64_t e = s.exp + head_exp;
                    scale_at[j] = e;
                    ka[j] = s.off >= 0 ? c.k_exp[e] : 127u;
                    ve[j] = s.off >= 0 ? c.v_exp[e] : 256u;
                } else {
                    if (lane == 0) *reinterpret_cast<uint32_t*>(my + fill * C::kStage + 2 * C::kTile + 4 * j) = some[j];
                }
            }
            constexpr int kStep = 32 / C::kChunks;  // rows a copy instruction of the warp covers
            if (sixteens && !kE2m1) {  // 16 keys lie after one another in a page: the address of one tells the others'
#pragma unroll
                for (int r = 0; r < kKeys; r += 16) {
                    const uint32_t there = (some[r / 32] >> (r & 31)) & 0xffffu;
                    const int one = there ? __ffs(there) - 1 : 0;
                    int64_t o = __shfl_sync(0xffffffffu, off[r / 32], (r & 31) + one) - one * c.slot_stride + lane_off;
                    if (!there) o = 0;
                    const char *ks = kbase + o, *vs = vbase + o;
#pragma unroll
                    for (int i = 0; i < 16; i += kStep) {
                        const int bytes = (there >> (i + lane / C::kChunks)) & 1u ? lane_bytes : 0;
                        const uint32_t dst = st + swizzle<C::kChunks>(r + i + lane / C::kChunks, lane % C::kChunks) * 16;
                        cp_async16<C::kHalfLines>(dst, ks, bytes, half_lines);
                        cp_async16<C::kHalfLines>(dst + C::kTile, vs, bytes, half_lines);
                        ks += rows_off;
                        vs += rows_off;
                    }
                }
            } else {  // unrolled by 4: e4m3, pages of one key, 74.9 -> 73.2 us; bf16 519 -> 511
#pragma unroll 4
                for (int r = 0; r < kKeys; r += kStep) {
                    const int row = r + lane / C::kChunks;
                    int64_t o = __shfl_sync(0xffffffffu, off[0], row & 31);
                    if constexpr (C::kLooks > 1) {
                        const int64_t o1 = __shfl_sync(0xffffffffu, off[C::kLooks - 1], row & 31);
                        if (row >= 32) o = o1;
                    }
                    const int bytes = o >= 0 ? lane_bytes : 0;
                    const int64_t at = bytes ? o + lane % C::kChunks * 16 : 0;
                    const uint32_t dst = st + swizzle<C::kChunks>(row, lane % C::kChunks) * 16;
                    cp_async16<C::kHalfLines>(dst, kbase + at, bytes, half_lines);
                    cp_async16<C::kHalfLines>(dst + C::kTile, vbase + at, bytes, half_lines);
                }
            }
            if constexpr (kE2m1) load_scales(st + 2 * C::kTile + C::kInfo, some, scale_at);
            info_stage = fill;
        }
        cp_async_commit();
        fill = fill + 1 == S ? 0 : fill + 1;
    };
    // e2m1, by sixteens, before a block of keys key0 .. of the range is used: its info from the bytes of its powers of two (0:
    // the page is not there); rows of d / 16 scale bytes to kScaleRow; and zeros for the scales and the power of two of keys that do
    // not count, so that whatever lies there (a NaN, a byte of 255) leaves them a product of zero and a score of -infinity.
    auto tidy = [&](uint8_t* stage, int key0, const Range& range) {
        if constexpr (kE2m1) {
            if (!by_sixteens) return;
            const bool widen = D == 128 && c.d < D;
            bool counts[C::kLooks], all = true;
#pragma unroll
            for (int j = 0; j < C::kLooks; ++j) {
                const int r = lane + 32 * j, key = key0 + r;
                const uint32_t k = stage[C::kExps + r], v = stage[C::kExps + kKeys + r];
                counts[j] = v != 0 && key >= range.first && key < range.len;
                all = all && counts[j];
                reinterpret_cast<float2*>(stage + 2 * C::kTile)[r] = make_float2(__uint_as_float(k << 23), counts[j] ? (float)((int)v - 127) : -INFINITY);
            }
            if (widen || __any_sync(0xffffffffu, !all)) {
                const uint32_t scales = smem_u32(stage) + 2 * C::kTile + C::kInfo;
                uint32_t w[C::kLooks][2][2];
                if (widen) {
#pragma unroll
                    for (int j = 0; j < C::kLooks; ++j)
#pragma unroll
                        for (int side = 0; side < 2; ++side) {
                            // 16 keys' rows of d / 16 bytes lie together at the beginning of their 16 kScaleRow bytes
                            const int r = lane + 32 * j;
                            const uint32_t from = scales + side * C::kScales + r / 16 * (16 * C::kScaleRow) + r % 16 * (c.d / 16);
                            w[j][side][0] = ld_shared_u16(from) | ld_shared_u16(from + 2) << 16;
                            w[j][side][1] = ld_shared_u16(from + 4);
                        }
                    __syncwarp();
                }
#pragma unroll
                for (int j = 0; j < C::kLooks; ++j) {
                    if (!widen && counts[j]) continue;
                    if (!counts[j]) reinterpret_cast<float2*>(stage + 2 * C::kTile)[lane + 32 * j].x = 0.f;
#pragma unroll
                    for (int side = 0; side < 2; ++side) {
                        const uint32_t to = scales + side * C::kScales + (lane + 32 * j) * C::kScaleRow;
                        const bool keep = widen && counts[j];
                        if constexpr (D == 128) st_shared_v2(to, keep ? w[j][side][0] : 0, keep ? w[j][side][1] : 0);
                        else if constexpr (D == 64) st_shared_u32(to, 0);
                        else st_shared_u16(to, 0);
                    }
                }
            }
            __syncwarp();
        }
    };
    auto store_info = [&]() {  // codes: the key's scale, and the value scale's exponent (-infinity: masked)
        if constexpr (kCodes) {
            if (info_stage < 0) return;
#pragma unroll
            for (int j = 0; j < C::kLooks; ++j)
                reinterpret_cast<float2*>(my + info_stage * C::kStage + 2 * C::kTile)[lane + 32 * j] =
                    make_float2(__uint_as_float(ka[j] << 23), ve[j] < 256 ? (float)((int)ve[j] - 127) : -INFINITY);
            info_stage = -1;
        }
    };
    // q of an item: thread (row, 16 elements); read while the first keys are on their way
    constexpr int kParts = D / 16;
    const int q_row = threadIdx.x / kParts, q_part = threadIdx.x % kParts;
    uint4 q_lo, q_hi;
    auto fetch_q = [&](const Segment& s) {
        const int hb = s.item % hblocks, head = (kPerHead ? s.b % c.hkv : s.item / hblocks) * group + hb * kRows + q_row;
        const int b = kPerHead ? s.b / c.hkv : s.b;
        const bool on = q_row < min(kRows, group - hb * kRows);
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + b * p.q_batch + (int64_t)head * p.q_head + 16 * q_part;
        q_lo = q_hi = make_uint4(0, 0, 0, 0);
        if (on && 16 * q_part < c.d) q_lo = *reinterpret_cast<const uint4*>(src);
        if (on && 16 * q_part + 8 < c.d) q_hi = *reinterpret_cast<const uint4*>(src + 8);
    };
    if constexpr (C::kSixteens && D == 128) {
        // d = 96: load_sixteens leaves V's last pieces out, which the look for rows of zeros takes as they are
        if (c.d < D)
            for (int i = lane; i < S * kKeys; i += 32)
                *reinterpret_cast<uint4*>(my + i / kKeys * C::kStage + C::kTile + swizzle<C::kChunks>(i % kKeys, C::kChunks - 1) * 16) = make_uint4(0, 0, 0, 0);
    }
    look();
    if (live) fetch_q(seg);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        load();
        look();
        store_info();
    }

    if constexpr (!kCluster) empty_rows();

    uint8_t* q_smem = smem + C::kRing;
    float* merge = reinterpret_cast<float*>(smem + C::kRing + C::kQ);
    float* q_scale = reinterpret_cast<float*>(smem + C::kRing + C::kQ + C::kMerge);
    const uint32_t q_addr = smem_u32(q_smem);
    const int g = lane >> 2, t = lane & 3;  // row and column group in the products' fragments
    int number = 0, use = 0;                // the segment's number, the stage to use next
    bool first_item = true;
    Torn ends_later{0, 0, 0, 0};
    // e2m1: where a lane's codes of K's row g and V's rows 2t, 2t+1 lie in a tile, V's scales (rows 8 and 16 further the same)
    const int row_key = kE2m1 ? key_of<D>(g) : g;
    uint32_t k_at = 0, v_at[2] = {0, 0}, vs_at[2] = {0, 0};
    if constexpr (kE2m1) {
        k_at = swizzle<C::kChunks>(row_key, D / 8 * t / 16) * 16 + D / 8 * t % 16;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int key = key_of<D>(2 * t + n);
            v_at[n] = swizzle<C::kChunks>(key, D / 16 * g / 16) * 16 + D / 16 * g % 16;
            vs_at[n] = key * C::kScaleRow + D / 8 * g / 16;
        }
    }

    for (; live; ++number) {
        const int hk = seg.item / hblocks, hb = seg.item % hblocks;
        const int head0 = hk * group + hb * kRows;        // first query head (kPerHead: of the sequence's group)
        const int rows = min(kRows, group - hb * kRows);  // query heads of the item

        // ---- q into shared memory, by whole warps (they exchange)
        if (threadIdx.x < (kRows * kParts + 31) / 32 * 32) {
            const int r = q_row, part = q_part;
            uint32_t w[8] = {q_lo.x, q_lo.y, q_lo.z, q_lo.w, q_hi.x, q_hi.y, q_hi.z, q_hi.w};
            float scale = p.scale * 1.4426950408889634f;
            if constexpr (kBf16 && kCodes) {
                float a = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    a = fmaxf(a, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
#pragma unroll
                for (int off = kParts / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
                // 2^n with a 2^-n in [2^14, 2^15): half's range then reaches 2^-38 of the largest element
                int n = (int)(__float_as_uint(a) >> 23) - 127 - 14;
                if (a == 0.f || !(a < INFINITY)) n = 0;
                if (n < -126) n = -126;
                const float up = __uint_as_float((uint32_t)(127 - n) << 23);
                scale *= __uint_as_float((uint32_t)(127 + n) << 23);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = pack2<false>(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
            }
            // 8-bit cache: elements 4t .. 4t+3 of 16 as columns 2t, 2t+1, 2t+8, 2t+9, the order its codes come in
            if (r < kRows) {
                uint4* row = reinterpret_cast<uint4*>(q_smem);
                row[swizzle<D / 8>(r, 2 * part)] = kE4m3 ? make_uint4(w[0], w[2], w[4], w[6]) : make_uint4(w[0], w[1], w[2], w[3]);
                row[swizzle<D / 8>(r, 2 * part + 1)] = kE4m3 ? make_uint4(w[1], w[3], w[5], w[7]) : make_uint4(w[4], w[5], w[6], w[7]);
                if (part == 0) q_scale[r] = scale;
            }
        }
        __syncthreads();
        // q as the first product's right operand: head g (+ 8), elements 2t, 2t+1 (and + 8) of 16
        uint32_t qf[kTiles][D / 16][2];
        float qscale[kTiles][2];
#pragma unroll
        for (int h = 0; h < kTiles; ++h) {
#pragma unroll
            for (int kk = 0; kk < D / 16; kk += 2) {
                uint32_t q4[4];
                if constexpr (kE2m1) {  // 8 elements for each 8 of the lane's codes, 4 of them a step
                    const uint4 x = ld_shared_v4(q_addr + swizzle<D / 8>(8 * h + g, D / 32 * t + kk / 2) * 16);
                    q4[0] = x.x, q4[1] = x.y, q4[2] = x.z, q4[3] = x.w;
                } else {
                    ldsm4(q_addr + swizzle<D / 8>(8 * h + (lane & 7), 2 * kk + (lane >> 3)) * 16, q4);
                }
                qf[h][kk][0] = q4[0];
                qf[h][kk][1] = q4[1];
                qf[h][kk + 1][0] = q4[2];
                qf[h][kk + 1][1] = q4[3];
            }
            qscale[h][0] = q_scale[8 * h + 2 * t];
            qscale[h][1] = q_scale[8 * h + 2 * t + 1];
        }
        // codes: a product with q in half, 2^31 (e4m3) or 2^34 (e2m1) at most, times the key's scale (to 2^126) and the row's
        // (2^-126 to 2^113 and the softmax's) must not overflow on the way to a score that does not.
        // The scales are multiplied first, a row's of more than 1 last.
        bool large_q = false;
        if constexpr (kCodes) {
#pragma unroll
            for (int h = 0; h < kTiles; ++h)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    large_q |= qscale[h][n] > 1.f;
                    qscale[h][n] = fminf(qscale[h][n], 1.f);
                }
        }

        float o[D / 16][kTiles][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int h = 0; h < kTiles; ++h) o[i][h][0] = o[i][h][1] = o[i][h][2] = o[i][h][3] = 0.f;
        // of heads 2t, 2t+1 (+ 8); l over this lane's keys, in e4m3 relative to a maximum of its own
        float m[kTiles][2], l[kTiles][2], ml[kTiles][2];
#pragma unroll
        for (int h = 0; h < kTiles; ++h) {
            m[h][0] = m[h][1] = -INFINITY;
            l[h][0] = l[h][1] = 0.f;
            ml[h][0] = ml[h][1] = kNoScore;
        }

        int here = seg.range.base + (seg.k0 + turn(number)) * kKeys;  // the block's first key
        for (int i = count(seg, number); i > 0; --i) {
            cp_async_wait<S - 2>();
            store_info();
            __syncwarp();
            tidy(my + use * C::kStage, here, seg.range);
            here += kWarps * kKeys;
            load();
            look();
            const uint32_t kt = my_addr + use * C::kStage, vt = kt + C::kTile;
            const uint8_t* info = my + use * C::kStage + 2 * C::kTile;
            use = use + 1 == S ? 0 : use + 1;
            // ---- scores, 16 keys at a time: keys g, g + 8 x heads 2t, 2t+1
            float sc[kMt][kTiles][4];
#pragma unroll
            for (int j = 0; j < kMt; ++j)
#pragma unroll
                for (int h = 0; h < kTiles; ++h) sc[j][h][0] = sc[j][h][1] = sc[j][h][2] = sc[j][h][3] = 0.f;
            if constexpr (!kCodes) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int j = 0; j < kMt; ++j) {
                        uint32_t k4[4];  // (keys 0-7, 8-15) of d 0-7, of d 8-15 of this step
                        ldsm4(kt + swizzle<C::kChunks>(16 * j + (lane & 15), 2 * kk + (lane >> 4)) * 16, k4);
#pragma unroll
                        for (int h = 0; h < kTiles; ++h) mma16816<kMmaBf16>(sc[j][h], k4, qf[h][kk][0], qf[h][kk][1]);
                    }
            } else if constexpr (kE2m1) {
#pragma unroll
                for (int j = 0; j < kMt; ++j) {
                    uint32_t ks[2][D / 32], kw[2][D / 32];  // of the keys of rows g, g + 8
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = 16 * j + 8 * e;
                        key_scales<D>(vt + C::kTile + C::kInfo + (key + row_key) * C::kScaleRow, t, ks[e]);
                        lane_codes<D, false>(kt + key * C::kRowBytes + k_at, kw[e]);
                    }
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) {
                        uint32_t a[4], b[4];
                        e2m1x8_to_f16x8(kw[0][w], a);
                        e2m1x8_to_f16x8(kw[1][w], b);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint32_t a4[4] = {hmul2(a[2 * m], ks[0][w]), hmul2(b[2 * m], ks[1][w]), hmul2(a[2 * m + 1], ks[0][w]),
                                                    hmul2(b[2 * m + 1], ks[1][w])};
#pragma unroll
                            for (int h = 0; h < kTiles; ++h) mma16816<false>(sc[j][h], a4, qf[h][2 * w + m][0], qf[h][2 * w + m][1]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < D / 16; kk += 2)
#pragma unroll
                    for (int j = 0; j < kMt; ++j) {
                        uint32_t k4[4];  // (keys 0-7, 8-15) of 16 codes, of the next 16: codes 4t .. 4t+3
                        ldsm4(kt + swizzle<C::kChunks>(16 * j + (lane & 15), kk + (lane >> 4)) * 16, k4);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t a4[4];
                            e4m3x4_to_f16x4(k4[2 * e], a4[0], a4[2]);
                            e4m3x4_to_f16x4(k4[2 * e + 1], a4[1], a4[3]);
#pragma unroll
                            for (int h = 0; h < kTiles; ++h) mma16816<false>(sc[j][h], a4, qf[h][kk + e][0], qf[h][kk + e][1]);
                        }
                    }
            }
            // ---- with codes s, and l; x, the running maximum, P
            if constexpr (kCodes) {
                float ev[kMt][2];  // of keys g, g + 8: the value scale's exponent, -infinity: masked
#pragma unroll
                for (int j = 0; j < kMt; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 f = reinterpret_cast<const float2*>(info)[16 * j + 8 * e + row_key];
                        ev[j][e] = f.y;
                        const float off = f.y == -INFINITY ? -INFINITY : 0.f;
#pragma unroll
                        for (int h = 0; h < kTiles; ++h)
#pragma unroll
                            for (int n = 0; n < 2; ++n) sc[j][h][2 * e + n] = fmaf(sc[j][h][2 * e + n], f.x * qscale[h][n], off);
                    }
                if (large_q) {
#pragma unroll
                    for (int h = 0; h < kTiles; ++h)
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const float rest = fmaxf(q_scale[8 * h + 2 * t + n], 1.f);
#pragma unroll
                            for (int j = 0; j < kMt; ++j) {
                                sc[j][h][n] *= rest;
                                sc[j][h][2 + n] *= rest;
                            }
                        }
                }
#pragma unroll
                for (int h = 0; h < kTiles; ++h)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        float mx = fmaxf(sc[0][h][n], sc[0][h][2 + n]);
#pragma unroll
                        for (int j = 1; j < kMt; ++j) mx = fmax3(mx, sc[j][h][n], sc[j][h][2 + n]);
                        if (mx - ml[h][n] > kRescale) {  // mx -infinity: not
                            l[h][n] *= ex2_approx(ml[h][n] - mx);
                            ml[h][n] = mx;
                        }
#pragma unroll
                        for (int j = 0; j < kMt; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                l[h][n] += ex2_approx(sc[j][h][2 * e + n] - ml[h][n]);
                                sc[j][h][2 * e + n] += ev[j][e];
                            }
                    }
            } else {
#pragma unroll
                for (int j = 0; j < kMt; ++j)
#pragma unroll
                    for (int h = 0; h < kTiles; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[j][h][e] *= qscale[0][0];
#pragma unroll
                for (int w = 0; w < C::kLooks; ++w) {
                    const uint32_t counts = reinterpret_cast<const uint32_t*>(info)[w];
                    if (counts != 0xffffffffu) {
#pragma unroll
                        for (int j = 2 * w; j < kMt && j < 2 * w + 2; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (!((counts >> (16 * (j - 2 * w) + 8 * e + g)) & 1u)) {
#pragma unroll
                                    for (int h = 0; h < kTiles; ++h) sc[j][h][2 * e] = sc[j][h][2 * e + 1] = -INFINITY;
                                }
                    }
                }
            }
            float mx[kTiles][2];
            auto grows = [&]() {  // this lane's maxima of the block; whether any lane's is well above the running maximum
                bool grow = false;
#pragma unroll
                for (int h = 0; h < kTiles; ++h)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mx[h][n] = fmaxf(sc[0][h][n], sc[0][h][2 + n]);
#pragma unroll
                        for (int j = 1; j < kMt; ++j) mx[h][n] = fmax3(mx[h][n], sc[j][h][n], sc[j][h][2 + n]);
                        grow |= mx[h][n] - m[h][n] > kRescale + kLift;  // exact where it matters; m + kRescale is not, past 2^26
                    }
                return __any_sync(0xffffffffu, grow);
            };
            bool grow = grows();
            if constexpr (kCodes) {
                // Looked for only where a maximum would grow: the first blocks, and rows of zeros that
                // stand out. (For every block it would be the stage's values read once more.)
                if (grow) {
                    uint32_t zeros[C::kLooks];  // as bits: keys that count, whose value codes are all 0
                    uint32_t some = 0;
#pragma unroll
                    for (int j = 0; j < C::kLooks; ++j) {
                        const int r = lane + 32 * j;
                        uint32_t any = 0;
#pragma unroll
                        for (int i = 0; i < C::kChunks; ++i) {
                            const uint4 w = *reinterpret_cast<const uint4*>(info - C::kTile + swizzle<C::kChunks>(r, i) * 16);
                            any |= w.x | w.y | w.z | w.w;
                        }
                        const bool counts = reinterpret_cast<const float2*>(info)[r].y > -INFINITY;
                        zeros[j] = __ballot_sync(0xffffffffu, counts && (any & (kE2m1 ? 0x77777777u : 0x7f7f7f7fu)) == 0);
                        some |= zeros[j];
                    }
                    if (some) {
#pragma unroll
                        for (int j = 0; j < kMt; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if ((zeros[j / 2] >> (16 * (j % 2) + 8 * e + row_key)) & 1u) {
#pragma unroll
                                    for (int h = 0; h < kTiles; ++h) sc[j][h][2 * e] = sc[j][h][2 * e + 1] = -INFINITY;
                                }
                        grow = grows();
                    }
                }
            }
            if (grow) {
#pragma unroll
                for (int h = 0; h < kTiles; ++h)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) mx[h][n] = fmaxf(mx[h][n], __shfl_xor_sync(0xffffffffu, mx[h][n], off));
                        const float m_new = fmaxf(m[h][n], mx[h][n] - kLift);
                        const float f = m_new == -INFINITY ? 1.f : ex2_approx(m[h][n] - m_new);
                        m[h][n] = m_new;
                        if constexpr (!kCodes) l[h][n] *= f;
#pragma unroll
                        for (int d = 0; d < D / 16; ++d) {
                            o[d][h][n] *= f;
                            o[d][h][2 + n] *= f;
                        }
                    }
            }
#pragma unroll
            for (int j = 0; j < kMt; ++j) {
                // P as the right operand: keys 2t, 2t+1 (and + 8) x head g; and the rest of its rounding,
                // together within 2^-16 (bfloat16) or 2^-22 (half) of a weight
                uint32_t pf[kTiles][2], pl[kTiles][2];
#pragma unroll
                for (int h = 0; h < kTiles; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            float& x = sc[j][h][2 * e + n];
                            x = ex2_approx(x - (m[h][n] == -INFINITY ? 0.f : m[h][n]));
                            if constexpr (!kCodes) l[h][n] += x;
                        }
                        const uint32_t w = pack2<kMmaBf16>(sc[j][h][2 * e], sc[j][h][2 * e + 1]);
                        pf[h][e] = transpose8(w);
                        if constexpr (!kRest) continue;
                        const float2 f = unpack2<kMmaBf16>(w);
                        pl[h][e] = transpose8(pack2<kMmaBf16>(sc[j][h][2 * e] - f.x, sc[j][h][2 * e + 1] - f.y));
                    }
                // ---- O^T += V^T P^T
                if constexpr (!kCodes) {
                    const int r = 16 * j + (lane & 7) + (lane & 16 ? 8 : 0);
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        uint32_t v4[4];  // keys 0-7 of (d 0-7, 8-15 of this tile), then keys 8-15
                        ldsm4_t(vt + swizzle<C::kChunks>(r, 2 * d + ((lane >> 3) & 1)) * 16, v4);
#pragma unroll
                        for (int h = 0; h < kTiles; ++h) {
                            mma16816<kMmaBf16>(o[d][h], v4, pf[h][0], pf[h][1]);
                            if constexpr (kRest) mma16816<kMmaBf16>(o[d][h], v4, pl[h][0], pl[h][1]);
                        }
                    }
                } else if constexpr (kE2m1) {
                    // rows 2t, 2t+1 (and + 8): the keys' scale as a pair, the codes as bytes of one key's and the other's
                    const uint32_t sc_at = vt + C::kTile + C::kInfo + C::kScales + 16 * j * C::kScaleRow;
                    constexpr int kVw = (D + 63) / 64;
                    uint32_t vs[2], even[2][kVw], odd[2][kVw];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t s = sc_at + 8 * e * C::kScaleRow;
                        vs[e] = e4m3x2_to_f16x2(ld_shared_u8(s + vs_at[0]) + ld_shared_u8(s + vs_at[1]) * 256u);
                        uint32_t a[kVw], b[kVw];
                        lane_codes<D, true>(vt + (16 * j + 8 * e) * C::kRowBytes + v_at[0], a);
                        lane_codes<D, true>(vt + (16 * j + 8 * e) * C::kRowBytes + v_at[1], b);
#pragma unroll
                        for (int w = 0; w < kVw; ++w) {
                            even[e][w] = (a[w] & 0x0f0f0f0fu) | ((b[w] << 4) & 0xf0f0f0f0u);
                            odd[e][w] = ((a[w] >> 4) & 0x0f0f0f0fu) | (b[w] & 0xf0f0f0f0u);
                        }
                    }
#pragma unroll
                    for (int w = 0; w < kVw; ++w) {  // rows g: the even codes, rows g + 8: the odd ones
                        uint32_t x[2][4], y[2][4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            e2m1x8_to_f16x8(even[e][w], x[e]);
                            e2m1x8_to_f16x8(odd[e][w], y[e]);
                        }
#pragma unroll
                        for (int i = 0; i < 4 && 4 * w + i < D / 16; ++i) {
                            const uint32_t a4[4] = {hmul2(x[0][i], vs[0]), hmul2(y[0][i], vs[0]), hmul2(x[1][i], vs[1]), hmul2(y[1][i], vs[1])};
#pragma unroll
                            for (int h = 0; h < kTiles; ++h) {
                                mma16816<false>(o[4 * w + i][h], a4, pf[h][0], pf[h][1]);
                                if constexpr (kRest) mma16816<false>(o[4 * w + i][h], a4, pl[h][0], pl[h][1]);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int d = 0; d < D / 16; d += 2) {
                        uint32_t v4[4];  // (keys 0-7, 8-15) of 16 codes, of the next 16: keys 2t, 2t+1 x codes 2g, 2g+1
                        ldsm4_t(vt + swizzle<C::kChunks>(16 * j + (lane & 15), d + (lane >> 4)) * 16, v4);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t a4[4];  // rows g: the even codes, rows g + 8: the odd ones
                            e4m3x4_to_f16x4(__byte_perm(v4[2 * e], 0, 0x3120), a4[0], a4[1]);
                            e4m3x4_to_f16x4(__byte_perm(v4[2 * e + 1], 0, 0x3120), a4[2], a4[3]);
#pragma unroll
                            for (int h = 0; h < kTiles; ++h) {
                                mma16816<false>(o[d + e][h], a4, pf[h][0], pf[h][1]);
                                if constexpr (kRest) mma16816<false>(o[d + e][h], a4, pl[h][0], pl[h][1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();  // the stage may be filled again
        }

        // ---- the warps' results together, kMergeRows rows at a time: a warp or two per row
        const bool whole = kCluster ? ranks == 1 : seg.k0 == 0 && seg.k1 == seg.nb;
        const int which = first_item ? 0 : 1;
        const int64_t out_row = (int64_t)seg.b * (kPerHead ? group : p.heads) + head0;
        // where the CTA's share of an item goes: for a cluster the ring, which is done with
        float* part = kCluster ? reinterpret_cast<float*>(smem) : partial<D, kRows>(p.workspace, blockIdx.x, which);
        if constexpr (kCluster) cp_async_wait<0>();
        else if (seg.k0 == 0 && !whole) ends_later = {rows, split.owner(seg.next - 1), which, (int)out_row};
#pragma unroll
        for (int h = 0; h < kTiles; ++h)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    float l2 = __shfl_xor_sync(0xffffffffu, l[h][n], off);
                    if constexpr (kCodes) {
                        const float ml2 = __shfl_xor_sync(0xffffffffu, ml[h][n], off), big = fmaxf(ml[h][n], ml2);
                        l[h][n] *= ex2_approx(ml[h][n] - big);
                        l2 *= ex2_approx(ml2 - big);
                        ml[h][n] = big;
                    }
                    l[h][n] += l2;
                }
#pragma unroll
        for (int round = 0; round < kRows / kMR; ++round) {  // rows kMR round ..; lane t has heads 2t, 2t+1 (+ 8)
            if (kMR * round >= rows) break;
            const int h = round * kMR / 8;
            if (t / (kMR / 2) == round % (8 / kMR)) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float* row = merge + (warp * kMR + 2 * (t % (kMR / 2)) + n) * C::kPitch;
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        if constexpr (!kCodes) {
                            row[16 * d + g] = o[d][h][n];
                            row[16 * d + 8 + g] = o[d][h][2 + n];
                        } else if constexpr (kE2m1) {
                            *reinterpret_cast<float2*>(row + D / 8 * g + 2 * d) = make_float2(o[d][h][n], o[d][h][2 + n]);
                        } else {
                            *reinterpret_cast<float2*>(row + 16 * d + 2 * g) = make_float2(o[d][h][n], o[d][h][2 + n]);
                        }
                    }
                    if (g == 0) *reinterpret_cast<Stats*>(row + D) = Stats{m[h][n], l[h][n], kCodes ? ml[h][n] : m[h][n], 0.f};
                }
            }
            __syncthreads();
            constexpr int kShare = kMR < kWarps ? kWarps / kMR : 1;  // warps per row
#pragma unroll
            for (int n = warp / kShare; n < kMR; n += kWarps / kShare) {
                const int r = kMR * round + n;
                if (r >= rows) break;
                float big = -INFINITY, big_l = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const Stats s = *reinterpret_cast<const Stats*>(merge + (w * kMR + n) * C::kPitch + D);
                    big = fmaxf(big, s.m);
                    big_l = fmaxf(big_l, s.ml);
                }
                float f[kWarps], sum = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const Stats s = *reinterpret_cast<const Stats*>(merge + (w * kMR + n) * C::kPitch + D);
                    const Factors<kCodes> to(s, big, big_l);
                    f[w] = to.o;
                    sum += to.l * s.l;
                }
                const Last<kCodes> last(big, big_l, sum);
#pragma unroll
                for (int d = lane + 32 * (warp % kShare); d < D; d += 32 * kShare) {
                    float a = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) a += f[w] * merge[(w * kMR + n) * C::kPitch + d];
                    if (!whole) part[r * D + d] = a;
                    else if (d < c.d) put<kBf16>(p.o, (out_row + r) * c.d + d, last(a));
                }
                if (lane == 0 && warp % kShare == 0) {
                    if (!whole) reinterpret_cast<Stats*>(part + kRows * D)[r] = Stats{big, sum, big_l, 0.f};
                    else p.lse[out_row + r] = last.lse;
                }
            }
            __syncthreads();
        }
        if constexpr (kCluster) {
            if (ranks > 1) join_cluster<D, kBf16, kCodes, kRows>(p, smem_u32(part), ranks, rank, rows, out_row);
            return;
        }
        first_item = false;
        live = seek(seg, seg.next);
        if (live) fetch_q(seg);
    }
    cp_async_wait<0>();
    if (threadIdx.x == 0) *torn<C, D>(p.workspace, blockIdx.x) = ends_later;
}

// Joins the items that several CTAs worked on: CTA (x, y) rows kJoinRows y .. of the item that
// begins in CTA x of the first kernel, if it ends in a later one. kShare warps a row, each for
// every kShare-th partial result, its lanes for the columns.
template <int D, bool kBf16, typename C, int kJoinRows>
__global__ void __launch_bounds__(kJoinThreads) fa2_decode_join_kernel(const DecodeParams p) {
    constexpr bool kCodes = C::kCodes;
    constexpr int kRows = C::kRows;
    constexpr int kShare = kJoinThreads / 32 / kJoinRows;
    constexpr int kCols = D / 32;  // columns a lane
    __shared__ float parts[kJoinThreads / 32][D];
    __shared__ Stats stats[kJoinThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_begin();
    const Torn item = *torn<C, D>(p.workspace, blockIdx.x);
    const int rows = item.rows;
    if ((int)blockIdx.y * kJoinRows >= rows) return;
    const int first = blockIdx.x, n = item.last_cta - first + 1, which = item.which;
    const int share = warp % kShare, r = blockIdx.y * kJoinRows + warp / kShare;
    const bool on = r < rows;
    float m = -INFINITY, ml = -INFINITY, l = 0.f, a[kCols] = {};
    if (on) {
#pragma unroll 4
        for (int k = share; k < n; k += kShare) {
            const float* s = partial<D, kRows>(p.workspace, first + k, k == 0 ? which : 0);
            const Stats st = reinterpret_cast<const Stats*>(s + kRows * D)[r];
            const Stats so_far{m, l, ml, 0.f};
            m = fmaxf(m, st.m);
            ml = fmaxf(ml, st.ml);
            const Factors<kCodes> old(so_far, m, ml), add(st, m, ml);
            l = l * old.l + add.l * st.l;
#pragma unroll
            for (int i = 0; i < kCols; ++i) a[i] = a[i] * old.o + add.o * s[r * D + lane + 32 * i];
        }
#pragma unroll
        for (int i = 0; i < kCols; ++i) parts[warp][lane + 32 * i] = a[i];
        if (lane == 0) stats[warp] = Stats{m, l, ml, 0.f};
    }
    __syncthreads();
    if (!on || share != 0) return;
    m = ml = -INFINITY;
#pragma unroll
    for (int w = 0; w < kShare; ++w) {
        m = fmaxf(m, stats[warp + w].m);
        ml = fmaxf(ml, stats[warp + w].ml);
    }
    float f[kShare];
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kShare; ++w) {
        const Stats st = stats[warp + w];
        const Factors<kCodes> to(st, m, ml);
        f[w] = to.o;
        l += to.l * st.l;
    }
    const Last<kCodes> last(m, ml, l);
    const int64_t row = (int64_t)item.out_row + r;
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
        const int d = lane + 32 * i;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kShare; ++w) v += f[w] * parts[warp + w][d];
        if (d < p.c.d) put<kBf16>(p.o, row * p.c.d + d, last(v));
    }
    if (lane == 0) p.lse[row] = last.lse;
}

// The cluster size of a call in one launch: the most CTAs per item, up to 8, with which all items'
// CTAs are resident at once. 0 where an item's blocks could be more than 4 for each of their warps
// (8 with more items than resident CTAs, which then balance one another): such a call goes by the
// lengths themselves, in two launches. GB300, 8 heads of d = 128, bf16, two launches against one:
// 1 sequence of 1000 8.5 / 6.7 us, of 2000 9.2 / 8.5; 30 of up to 200 11.0 / 8.8; 64 of up to 500
// (8 blocks a warp) 23.4 / 21.5; past the limit 8 of up to 2000 13.0 / 15.2 (8 blocks a warp).
//
// With a table for each key-value head all rows are as a rule equally long (what fa2_select_pages gives), which the two
// launches' division has nothing to add to: any number of CTAs that are resident at once, up to 16 blocks a warp.
template <typename C, bool kPerHead>
int cluster_ranks(const DecodeParams& p) {
    const int64_t keys = p.window > 0 && p.window + 15 < p.c.room ? p.window + 15 : p.c.room;
    const int64_t blocks = (keys + C::kKeys - 1) / C::kKeys;
    const int group = p.heads / p.c.hkv;
    const int64_t items = p.c.batch * p.seq_heads() * ((group + C::kRows - 1) / C::kRows);
    const int64_t resident = 152 * C::kShortPerSm;
    int ranks = 1;
    if constexpr (kPerHead) {
        ranks = (int)std::max<int64_t>(1, std::min<int64_t>({8, resident / items, (blocks + kWarps - 1) / kWarps}));
        return blocks <= (int64_t)ranks * kWarps * 16 && items * ranks <= INT32_MAX ? ranks : 0;
    }
    while (ranks < 8 && items * ranks * 2 <= resident && blocks > ranks * kWarps) ranks *= 2;
    const int64_t most = (int64_t)ranks * kWarps * (items > resident ? 8 : 4);
    return blocks <= most && items * ranks <= INT32_MAX ? ranks : 0;
}

template <int D, bool kBf16, int kForm, int kTiles, bool kPerHead>
cudaError_t launch_d(const DecodeParams& p, cudaStream_t stream, int slot) {
    using C = Cfg<D, kForm, kTiles>;
    int ranks = cluster_ranks<C, kPerHead>(p);
    if (ranks) {
        auto kern = fa2_decode_kernel<D, kBf16, kForm, kTiles, kPerHead, true>;
        cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), C::kSmem, slot + 1);
        if (e != cudaSuccess) return e;
        const int ask = ranks <= 2 ? ranks : (ranks <= 4 ? 4 : 8);
        if (ranks == 1 || cluster_fits(reinterpret_cast<const void*>(kern), kThreads, C::kSmem, ask, slot + 1)) {
            const int64_t items = p.c.batch * p.seq_heads() * ((p.heads / p.c.hkv + C::kRows - 1) / C::kRows);
            decode_record() = ranks;
            return launch_early_cluster(kern, dim3((unsigned)(items * ranks)), dim3(kThreads), C::kSmem, stream, (unsigned)ranks, p, ranks);
        }
    }
    decode_record() = 0;
    auto kern = fa2_decode_kernel<D, kBf16, kForm, kTiles, kPerHead, false>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), C::kSmem, slot);
    if (e != cudaSuccess) return e;
    e = launch_early(kern, dim3(C::kMaxCtas), dim3(kThreads), C::kSmem, stream, p, 1);
    if (e != cudaSuccess) return e;
    const int rows = std::min(C::kRows, p.heads / p.c.hkv);
    const int64_t items = p.c.batch * p.seq_heads() * ((p.heads / p.c.hkv + C::kRows - 1) / C::kRows);
    // The fewer rows an item has, and the fewer items (of more partial results each), the more warps
    // for a row. GB300: one key-value head, 100,000 tokens, 4 query heads 36 us with a quarter of the
    // warps for each row, 23 us with all; 8 heads 11.0 us with a quarter, 10.4 half, 11.8 all.
    auto join = [&](void (*kernel)(DecodeParams), int join_rows) {
        return launch_early(kernel, dim3(C::kMaxCtas, (unsigned)((rows + join_rows - 1) / join_rows)), dim3(kJoinThreads), 0, stream, p);
    };
    if (rows == 1 || items <= kFewItems) return join(fa2_decode_join_kernel<D, kBf16, C, 1>, 1);
    if (rows == 2 || items <= 2 * kFewItems) return join(fa2_decode_join_kernel<D, kBf16, C, 2>, 2);
    return join(fa2_decode_join_kernel<D, kBf16, C, 4>, 4);
}

// Up to 8 query heads a key-value head: one column tile, else two.
template <int D, bool kBf16, int kForm, bool kPerHead>
cudaError_t launch_tiles(const DecodeParams& p, cudaStream_t stream, int slot) {
    return p.heads / p.c.hkv <= 8 ? launch_d<D, kBf16, kForm, 1, kPerHead>(p, stream, slot)
                                   : launch_d<D, kBf16, kForm, 2, kPerHead>(p, stream, slot + 2);
}

// Rows of 16 bits and e4m3 codes; those of e2m1 codes are compiled apart (launch_e2m1).
template <int D, bool kPerHead>
cudaError_t launch_kind(const DecodeParams& p, cudaStream_t stream, int slot) {  // slots slot .. slot + 15
    const bool bf = p.c.dtype == kBf16;
    if (p.c.form == kRowsE4m3)
        return bf ? launch_tiles<D, true, kRowsE4m3, kPerHead>(p, stream, slot) : launch_tiles<D, false, kRowsE4m3, kPerHead>(p, stream, slot + 4);
    return bf ? launch_tiles<D, true, kRows16, kPerHead>(p, stream, slot + 8) : launch_tiles<D, false, kRows16, kPerHead>(p, stream, slot + 12);
}

template <int D, bool kPerHead>
cudaError_t launch_e2m1(const DecodeParams& p, cudaStream_t stream, int slot) {  // slots slot .. slot + 15
    if (p.by_sixteens)
        return p.c.dtype == kBf16 ? launch_tiles<D, true, kRowsE2m1By16, kPerHead>(p, stream, slot)
                                  : launch_tiles<D, false, kRowsE2m1By16, kPerHead>(p, stream, slot + 4);
    return p.c.dtype == kBf16 ? launch_tiles<D, true, kRowsE2m1, kPerHead>(p, stream, slot + 8)
                              : launch_tiles<D, false, kRowsE2m1, kPerHead>(p, stream, slot + 12);
}

template <int D, int kTiles>
size_t workspace_for(bool e2m1) {
    using C = Cfg<D, kRowsE4m3, kTiles>;
    const int ctas = e2m1 ? Cfg<D, kRowsE2m1, kTiles>::kMaxCtas : std::max(C::kMaxCtas, Cfg<D, kRows16, kTiles>::kMaxCtas);
    return (size_t)ctas * (2 * C::kRows * (D + 4) * sizeof(float) + sizeof(Torn));
}

}  // namespace
}  // namespace fa2
