// kv_select.cu - bounds of the keys in a page, and the pages whose keys can score highest for a query.
//
// Bounds: the lowest and the highest key of every channel, as 8-bit integers at a power of two of the page and
// head, rounded outwards: for 16 tokens of 128 channels in 16 bits 257 bytes for 8192 of keys and values.
//
// Scores: sum_c max(q_c low_c, q_c high_c) is no less than q . k for any key within the bounds. The query's
// 8-bit integers, split into those above zero (which meet the highest keys) and those below (the lowest), make it
// a sum of integer products: exact, so that which pages are taken does not depend on the order of sums, and a
// float32 holds the result (below 2^21) times powers of two.
//
// Selection: the budget-th largest score by counting, the earlier page first among equals, pages in the order of
// their positions.
#include <algorithm>

#include "paged.cuh"

namespace fa2 {
namespace {

constexpr int kWarps = 4;
constexpr int kMinExp = -60;

// e of the smallest power of two with a <= 127 2^e, at least -60; 0 for a = 0.
__device__ __forceinline__ int bound_exp(float a) {
    if (!(a > 0.f)) return 0;
    const uint32_t bits = __float_as_uint(a);
    const int k = (int)(bits >> 23) - 126;  // a = f 2^k, f in [1/2, 1): 127 = 127/128 2^7
    return max(k - 7 + ((bits & 0x7fffffu) > 0x7e0000u ? 1 : 0), kMinExp);
}
__device__ __forceinline__ float exp2_of(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }  // -126 <= e <= 127

// Pairs of keys' channels as 16-bit floats that hold them exactly: the cache's own type, or bfloat16 for codes.
template <bool kBf16>
struct Pair {
    using T = __nv_bfloat162;
};
template <>
struct Pair<false> {
    using T = __half2;
};
template <bool kBf16>
__device__ __forceinline__ float2 floats(uint32_t w) {
    if constexpr (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// A warp takes one page of one sequence and one head: groups of 16 lanes (kLanes) read slots in turn, 8 channels a lane.
template <bool kBf16, int kForm, int kLanes>
__global__ void __launch_bounds__(kWarps * 32) kv_bounds_kernel(const KvBoundsParams p) {
    const PagedParams& c = p.c;
    constexpr bool kPairBf16 = kBf16 || kForm != kRows16;
    using T = typename Pair<kPairBf16>::T;
    constexpr int kGroups = 32 / kLanes, kUnroll = 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
    const int h = blockIdx.y;
    grid_begin();
    // ---- which page: sequence b has room for n / page_size + 2 of them, its first is number cu_new[b] / page_size + 2 b
    int b, count = 1;
    int64_t nth = 0;
    if (p.cu_new) {
        auto start = [&](int i) { return (int64_t)page_of(c, max(p.cu_new[i], 0)) + 2 * i; };
        int lo = 0, hi = (int)c.batch;
        if (w >= start(hi)) return;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start(mid) <= w) lo = mid;
            else hi = mid;
        }
        b = lo;
        nth = w - start(b);
        count = p.cu_new[b + 1] - p.cu_new[b];
    } else {
        if (w >= c.batch) return;
        b = (int)w;
        if (c.lens[b] == 0) return;
    }
    if (count <= 0 || nth < 0) return;
    const int given = c.lens[b], len = bounded_len(given, c.room, c.status);
    int first = given - count;
    if (first < 0) {  // tokens without a position
        if (c.status && lane == 0) atomicOr(c.status, kStatusBadIndex);
        first = 0;
    }
    if (first >= len) return;
    const int64_t j = page_of(c, first) + nth;
    if (j * c.page_size >= len) return;
    const Slot at = slot_of(c, c.table[b * c.table_stride + j], 0);
    if (at.off < 0) return;
    const int live = (int)min((int64_t)c.page_size, len - j * c.page_size);
    // ---- lowest and highest of the lane's channels
    const int li = lane % kLanes, gr = lane / kLanes;
    const bool on = 8 * li < c.d;
    constexpr uint32_t kInf2 = kPairBf16 ? 0x7f807f80u : 0x7c007c00u;
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) lo[i] = kInf2, hi[i] = kInf2 | 0x80008000u;
    auto widen = [&](uint32_t word) { return *reinterpret_cast<T*>(&word); };
    auto bits = [&](T x) { return *reinterpret_cast<uint32_t*>(&x); };
    const char* base = c.k + at.off + h * c.head_stride;
    const int64_t exp0 = at.exp + (int64_t)h * c.page_size;
    for (int s0 = gr; s0 < live; s0 += kGroups * kUnroll) {
        uint32_t k[kUnroll][4];
        uint32_t byte[kUnroll], scale[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int s = s0 + u * kGroups;
            if (s >= live || !on) continue;
            const char* row = base + s * c.slot_stride;
            if constexpr (kForm == kRows16) {
                const uint4 x = *reinterpret_cast<const uint4*>(row + 16 * li);
                k[u][0] = x.x, k[u][1] = x.y, k[u][2] = x.z, k[u][3] = x.w;
            } else if constexpr (kForm == kRowsE4m3) {
                const uint2 x = *reinterpret_cast<const uint2*>(row + 8 * li);
                k[u][0] = x.x, k[u][1] = x.y;
                byte[u] = c.k_exp[exp0 + s];
            } else {
                k[u][0] = *reinterpret_cast<const uint32_t*>(row + 4 * li);
                byte[u] = c.k_exp[exp0 + s];
                scale[u] = c.k_scale[(exp0 + s) * (c.d / 16) + li / 2];
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (s0 + u * kGroups >= live || !on) continue;
            uint32_t x[4];
            if constexpr (kForm == kRows16) {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = k[u][i];
            } else {
                uint32_t f[4];
                if constexpr (kForm == kRowsE4m3) {
                    e4m3x4_to_f16x4(k[u][0], f[0], f[1]);
                    e4m3x4_to_f16x4(k[u][1], f[2], f[3]);
                } else {
                    e2m1x8_to_f16x8(k[u][0], f);
                    const uint32_t s = e4m3x2_to_f16x2(scale[u] * 0x101u);
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = hmul2(f[i], s);
                }
                const float two = __uint_as_float(byte[u] << 23);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
                    x[i] = pack2<true>(y.x * two, y.y * two);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // (a NaN is not taken)
                lo[i] = bits(__hmin2(widen(lo[i]), widen(x[i])));
                hi[i] = bits(__hmax2(widen(hi[i]), widen(x[i])));
            }
        }
    }
#pragma unroll
    for (int off = kLanes; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = bits(__hmin2(widen(lo[i]), widen(__shfl_xor_sync(0xffffffffu, lo[i], off))));
            hi[i] = bits(__hmax2(widen(hi[i]), widen(__shfl_xor_sync(0xffffffffu, hi[i], off))));
        }
    // ---- codes
    float l[8], u[8], a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = floats<kPairBf16>(lo[i]), y = floats<kPairBf16>(hi[i]);
        l[2 * i] = x.x, l[2 * i + 1] = x.y, u[2 * i] = y.x, u[2 * i + 1] = y.y;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (l[i] > u[i]) l[i] = u[i] = 0.f;  // nothing but NaN
        const float x = fabsf(l[i]), y = fabsf(u[i]);
        a = fmaxf(a, fmaxf(x < INFINITY ? x : 0.f, y < INFINITY ? y : 0.f));
    }
    if (!on) a = 0.f;
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
    const int e = bound_exp(a);
    if (gr != 0 || !on) return;
    const float inv = exp2_of(-e);
    uint32_t out[2][2] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int low = (int)fmaxf(fminf(floorf(l[i] * inv), 127.f), -127.f), high = (int)fmaxf(fminf(ceilf(u[i] * inv), 127.f), -127.f);
        out[0][i / 4] |= (uint32_t)(low & 0xff) << (8 * (i % 4));
        out[1][i / 4] |= (uint32_t)(high & 0xff) << (8 * (i % 4));
    }
    const int64_t row = at.exp / c.page_size + h;  // page * hkv + h
    int8_t* dst = p.bounds + row * 2 * c.d + 8 * li;
    *reinterpret_cast<uint2*>(dst) = make_uint2(out[0][0], out[0][1]);
    *reinterpret_cast<uint2*>(dst + c.d) = make_uint2(out[1][0], out[1][1]);
    if (li == 0) p.bounds_exp[row] = (uint8_t)(e + 127);
}

template <bool kBf16, int kForm>
cudaError_t launch_bounds_form(const KvBoundsParams& p, cudaStream_t stream) {
    const int64_t pages = p.cu_new ? p.tokens / p.c.page_size + 2 * p.c.batch : p.c.batch;
    const dim3 grid((unsigned)((pages + kWarps - 1) / kWarps), (unsigned)p.c.hkv);
    if (p.c.d <= 32) return launch_early(kv_bounds_kernel<kBf16, kForm, 4>, grid, dim3(kWarps * 32), 0, stream, p);
    if (p.c.d <= 64) return launch_early(kv_bounds_kernel<kBf16, kForm, 8>, grid, dim3(kWarps * 32), 0, stream, p);
    return launch_early(kv_bounds_kernel<kBf16, kForm, 16>, grid, dim3(kWarps * 32), 0, stream, p);
}

// ---------------------------------------------------------------------------- scores

constexpr uint32_t kForced = 0xffffffffu;  // above every score's key; a page outside the cache: 0, below every score's
constexpr int kSets = 1;                   // times 16 pages a warp takes at once

// Unsigned numbers in the order of the floats (no NaN).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Pages that hold a length's keys.
__device__ __forceinline__ int pages_of(const SelectParams& p, int len) {
    if (len == 0) return 0;
    const uint32_t last = (uint32_t)len - 1;
    return (int)((__umulhi(p.page_mul, last) + last) >> p.page_shift) + 1;  // as page_of
}

// The scores of pages of one sequence and key-value head, as products of 16 pages' bounds with 8 heads' integers: a row of
// bounds is 2 d bytes, the lowest keys and then the highest, and meets the head's integers below zero and then those
// above. Lane 4 g + t reads the 16-byte pieces t, t + 4, ... of the rows g and g + 8 straight into the left operand (a
// product takes its 32 terms in any order, the right operand the same); kPieces of them. GB300, 16 sequences to 65536
// in pages of 32, 8 heads of 8: 6 us with them, 39 with four-term dot products and sums over lanes.
template <bool kBf16, int kPieces>
__global__ void __launch_bounds__(kWarps * 32) page_scores_kernel(const SelectParams p, int row_ctas) {
    constexpr int kRow = 64 * kPieces;  // bytes of a head's integers: [below zero][above], zeros behind 2 d
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int padded = (p.group + 7) / 8 * 8;
    float* const two = reinterpret_cast<float*>(smem + (size_t)padded * kRow);  // 2^e a head
    grid_begin();
    const int row = blockIdx.x / row_ctas, cta = blockIdx.x % row_ctas, b = row / p.hkv, hk = row % p.hkv;
    const int pages = pages_of(p, bounded_len(p.lens[b], p.per_seq * p.page_size, p.status));
    if (pages <= p.budget || (int64_t)cta * kWarps * 16 * kSets >= pages) return;  // all are taken; nothing left for this CTA
    // ---- the queries' integers: a warp a head, 4 channels a lane (d <= 128)
    for (int h = warp; h < padded; h += kWarps) {
        float x[4] = {}, a = 0.f;
        if (h < p.group && 4 * lane < p.d) {
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + b * p.q_batch +
                                                            ((int64_t)hk * p.group + h) * p.q_head + 4 * lane);
            const float2 f = floats<kBf16>(w.x), g = floats<kBf16>(w.y);
            x[0] = f.x, x[1] = f.y, x[2] = g.x, x[3] = g.y;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (x[i] != x[i]) x[i] = 0.f;
            a = fmaxf(a, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        const int e = bound_exp(a);
        const float inv = exp2_of(-e);
        uint32_t up = 0, down = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int q = (int)fmaxf(fminf(rintf(x[i] * inv), 127.f), -127.f);
            up |= (uint32_t)max(q, 0) << (8 * i);
            down |= (uint32_t)(min(q, 0) & 0xff) << (8 * i);
        }
        uint32_t* ints = reinterpret_cast<uint32_t*>(smem + h * kRow);
        if (4 * lane < p.d) {
            ints[lane] = down;
            ints[p.d / 4 + lane] = up;
        }
        for (int i = p.d / 2 + lane; i < kRow / 4; i += 32) ints[i] = 0;
        if (lane == 0) two[h] = h < p.group ? exp2_of(e) : 0.f;
    }
    __syncthreads();
    const int g = lane >> 2, t = lane & 3;
    const int32_t* table = p.table + b * p.table_stride;
    uint32_t* out = p.scores + (int64_t)row * p.per_seq;
    const int64_t step = (int64_t)row_ctas * kWarps * 16 * kSets;
    // lane r < 16 kSets looks page r of the warp's up
    auto look = [&](int64_t j) { return lane < 16 * kSets && j + lane < pages ? table[j + lane] : -1; };
    int64_t j0 = ((int64_t)cta * kWarps + warp) * 16 * kSets;
    int next = look(j0);
    for (; j0 < pages; j0 += step) {
        int64_t at = next >= 0 && next < p.num_pages ? (int64_t)next * p.hkv + hk : -1;
        const float scale = at >= 0 ? __uint_as_float((uint32_t)p.bounds_exp[at] << 23) : 0.f;
        if (at < 0 && lane < 16 * kSets && j0 + lane < pages && p.status) atomicOr(p.status, kStatusBadIndex);
        uint4 a[kSets][2][kPieces];
#pragma unroll
        for (int s = 0; s < kSets; ++s)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int64_t here = __shfl_sync(0xffffffffu, at, 16 * s + 8 * r + g);
                const int8_t* src = p.bounds + (here >= 0 ? here : 0) * 2 * p.d + 16 * t;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    a[s][r][i] = make_uint4(0, 0, 0, 0);
                    if (here >= 0 && 64 * i + 16 * t < 2 * p.d) a[s][r][i] = *reinterpret_cast<const uint4*>(src + 64 * i);
                }
            }
        next = look(j0 + step);
        float best[kSets][2];
#pragma unroll
        for (int s = 0; s < kSets; ++s) best[s][0] = best[s][1] = -INFINITY;
        for (int h0 = 0; h0 < padded; h0 += 8) {
            int c[kSets][4] = {};
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const uint4 q = *reinterpret_cast<const uint4*>(smem + (h0 + g) * kRow + 64 * i + 16 * t);
#pragma unroll
                for (int s = 0; s < kSets; ++s) {
                    mma_s8(c[s], a[s][0][i].x, a[s][1][i].x, a[s][0][i].y, a[s][1][i].y, q.x, q.y);
                    mma_s8(c[s], a[s][0][i].z, a[s][1][i].z, a[s][0][i].w, a[s][1][i].w, q.z, q.w);
                }
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {  // heads 2t, 2t+1
                if (h0 + 2 * t + n >= p.group) continue;
                const float f = two[h0 + 2 * t + n];
#pragma unroll
                for (int s = 0; s < kSets; ++s) {
                    best[s][0] = fmaxf(best[s][0], (float)c[s][n] * f);
                    best[s][1] = fmaxf(best[s][1], (float)c[s][2 + n] * f);
                }
            }
        }
        // ---- lane r has page r's score
        float mine = 0.f;
#pragma unroll
        for (int s = 0; s < kSets; ++s)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = best[s][r];
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                x = __shfl_sync(0xffffffffu, x, lane % 8 * 4);
                if (lane / 8 == 2 * s + r) mine = x;
            }
        const int64_t j = j0 + lane;
        if (lane < 16 * kSets && j < pages)
            out[j] = j < p.first || j >= pages - p.recent ? kForced : (at >= 0 ? ordered(mine * scale) : 0u);
    }
}

// ---------------------------------------------------------------------------- selection

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32, kBins = 2 * kSelThreads;

// Sums over the CTA of a thread's two counts, exclusive in thread order, and their totals.
__device__ __forceinline__ uint2 scan2(uint2 v, uint2* sums, uint2* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint2 upto = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, upto.x, off), y = __shfl_up_sync(0xffffffffu, upto.y, off);
        if (lane >= off) upto.x += x, upto.y += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    uint2 before = make_uint2(0, 0), all = before;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
        if (w < warp) before.x += sums[w].x, before.y += sums[w].y;
        all.x += sums[w].x, all.y += sums[w].y;
    }
    *total = all;
    return make_uint2(before.x + upto.x - v.x, before.y + upto.y - v.y);
}

// A CTA takes one sequence and head. Thread i has the scores of pages i per .. in registers, kHeld at most; more are read
// again. The budget-th largest is found by counting into kBins equal parts of the range that holds it, three times at
// the most (for 32 bits), mostly twice: the range begins as that of the scores there are.
template <int kHeld>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
    __shared__ uint2 sums[kSelWarps];
    __shared__ uint32_t bins[kBins];
    __shared__ uint32_t found[3];
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) found[0] = 0xffffffffu, found[1] = 0u, found[2] = 0u;
    grid_begin();
    const int b = blockIdx.x / p.hkv;
    const int len = bounded_len(p.lens[b], p.per_seq * p.page_size, p.status);
    const int n = pages_of(p, len);
    const int32_t* table = p.table + b * p.table_stride;
    int32_t* dst = p.sel_table + (int64_t)blockIdx.x * p.budget;
    const int taken = min(n, p.budget);
    for (int i = taken + threadIdx.x; i < p.budget; i += kSelThreads) dst[i] = -1;
    if (n <= p.budget) {
        for (int i = threadIdx.x; i < n; i += kSelThreads) {
            const int page = table[i];
            dst[i] = page;
            if ((page < 0 || page >= p.num_pages) && p.status) atomicOr(p.status, kStatusBadIndex);
        }
        if (threadIdx.x == 0) p.sel_lens[blockIdx.x] = len;
        return;
    }
    const uint32_t* scores = p.scores + (int64_t)blockIdx.x * p.per_seq;
    const int per = (n + kSelThreads - 1) / kSelThreads;
    const int i0 = (int)min((int64_t)threadIdx.x * per, (int64_t)n), mine = min(per, n - i0);
    const bool held = per <= kHeld;
    uint32_t key[kHeld];
    if (held) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            if (i < mine) key[i] = scores[i0 + i];
        }
    }
    auto each = [&](auto f) {
        if (held) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                if (i < mine) f(i0 + i, key[i]);
            }
        } else {
            for (int i = 0; i < mine; ++i) f(i0 + i, scores[i0 + i]);
        }
    };
    // ---- the range of the scores that are not forced, and how many to take of those
    uint32_t lo = 0xffffffffu, hi = 0, forced = 0;
    each([&](int, uint32_t k) {
        if (k == kForced) ++forced;
        else lo = min(lo, k), hi = max(hi, k);
    });
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    forced = __reduce_add_sync(0xffffffffu, forced);
    __syncthreads();  // found is set
    if (lane == 0) {
        atomicMin(&found[0], lo);
        atomicMax(&found[1], hi);
        if (forced) atomicAdd(&found[2], forced);
    }
    __syncthreads();
    lo = found[0], hi = found[1];
    uint32_t need = (uint32_t)p.budget - found[2];
    uint32_t least = kForced - 1, equal = 0;  // all above `least` are taken and the earliest `equal` of those equal to it
    while (need) {
        const uint32_t width = hi - lo;  // less one
        const int shift = max(0, 32 - __clz(width) - 10);
        bins[threadIdx.x] = bins[kSelThreads + threadIdx.x] = 0;
        __syncthreads();  // (found is read)
        each([&](int, uint32_t k) {
            if (k >= lo && k <= hi) atomicAdd(&bins[(k - lo) >> shift], 1u);
        });
        __syncthreads();
        // thread i has the parts i and i + 1 from the top, in pairs
        const int top = kBins - 1 - 2 * (int)threadIdx.x;
        const uint32_t c0 = bins[top], c1 = bins[top - 1];
        uint2 total;
        const uint32_t above = scan2(make_uint2(c0 + c1, 0), sums, &total).x;
        if (above < need && need <= above + c0 + c1) {
            const bool second = need > above + c0;
            found[0] = second ? top - 1 : top;
            found[1] = second ? above + c0 : above;
            found[2] = second ? c1 : c0;
        }
        __syncthreads();
        lo += found[0] << shift;
        hi = min(hi, lo + ((1u << shift) - 1));
        need -= found[1];
        least = lo;
        if (shift == 0 || need == found[2]) {
            equal = shift == 0 ? need : 0xffffffffu;  // (with the whole part: its lowest and all above)
            break;
        }
        if (lo == hi) {
            equal = need;
            break;
        }
    }
    // ---- in the order of their positions
    uint2 count = make_uint2(0, 0), total;
    each([&](int, uint32_t k) { count.x += k > least, count.y += k == least; });
    const uint2 before = scan2(count, sums, &total);
    uint32_t at = before.x + min(before.y, equal), seen = before.y;
    each([&](int i, uint32_t k) {
        const bool take = k > least || (k == least && seen < equal);
        seen += k == least;
        if (take) dst[at++] = table[i];
        if (i == n - 1) p.sel_lens[blockIdx.x] = p.budget * p.page_size - (take ? (int)((int64_t)n * p.page_size - len) : 0);
    });
}

template <bool kBf16, int kPieces>
cudaError_t launch_scores(const SelectParams& p, cudaStream_t stream) {
    const int padded = (p.group + 7) / 8 * 8;
    const size_t smem = (size_t)padded * (64 * kPieces + sizeof(float));  // 33 KB at most
    // As many CTAs for a sequence and head as fill the SMs kResident times over, at most one for each round of pages.
    constexpr int kPages = kWarps * 16 * kSets, kResident = 6;
    const int64_t rows = p.batch * p.hkv, most = (p.per_seq + kPages - 1) / kPages;
    const int64_t row_ctas = std::max<int64_t>(1, std::min(most, (152 * kResident + rows - 1) / rows));
    return launch_early(page_scores_kernel<kBf16, kPieces>, dim3((unsigned)(rows * row_ctas)), dim3(kWarps * 32), smem, stream, p, (int)row_ctas);
}

template <bool kBf16>
cudaError_t launch_scores_type(const SelectParams& p, cudaStream_t stream) {
    switch ((p.d + 31) / 32) {
        case 1: return launch_scores<kBf16, 1>(p, stream);
        case 2: return launch_scores<kBf16, 2>(p, stream);
        case 3: return launch_scores<kBf16, 3>(p, stream);
        default: return launch_scores<kBf16, 4>(p, stream);
    }
}

}  // namespace

cudaError_t launch_kv_bounds(const KvBoundsParams& p, cudaStream_t stream) {
    const bool bf = p.c.dtype == kBf16;
    switch (p.c.form) {
        case kRows16: return bf ? launch_bounds_form<true, kRows16>(p, stream) : launch_bounds_form<false, kRows16>(p, stream);
        case kRowsE4m3: return launch_bounds_form<true, kRowsE4m3>(p, stream);
        default: return launch_bounds_form<true, kRowsE2m1>(p, stream);
    }
}

cudaError_t launch_select_pages(const SelectParams& p, cudaStream_t stream) {
    if (p.per_seq > p.budget) {  // else every page is taken, without a look at the bounds
        const cudaError_t e = p.dtype == kBf16 ? launch_scores_type<true>(p, stream) : launch_scores_type<false>(p, stream);
        if (e != cudaSuccess) return e;
    }
    // (by the table's width: the lengths are on the device)
    auto kern = p.per_seq <= 4 * kSelThreads ? select_kernel<4> : select_kernel<16>;
    return launch_early(kern, dim3((unsigned)(p.batch * p.hkv)), dim3(kSelThreads), 0, stream, p);
}

}  // namespace fa2
