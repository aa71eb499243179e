// kv_select.cu - bounds of the keys in a page, and the pages whose keys can score highest for a query.
//
// Bounds: the lowest and the highest key of every channel, as 8-bit integers at a power of two of the page and
// head, rounded outwards: for 16 tokens of 128 channels in 16 bits 257 bytes for 8192 of keys and values.
//
// Scores: sum_c max(q_c low_c, q_c high_c) is no less than q . k for any key within the bounds. The query's
// 8-bit integers, split into those above zero (which meet the highest keys) and those below (the lowest), make it
// two sums of integer products, four to an instruction: exact, so that which pages are taken does not depend on
// the order of sums, and a float32 holds the result (below 2^21) times powers of two.
//
// Selection: the budget-th largest score by bisection on its bits, the earlier page first among equals, pages in
// the order of their positions.
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

constexpr int kHeads = 8;       // query heads whose integers a lane holds at a time
constexpr uint32_t kForced = 0xffffffffu;  // above every score's key; a page outside the cache: 0, below every score's

// Unsigned numbers in the order of the floats (no NaN).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ int dot4(uint32_t a, uint32_t b, int c) { return __dp4a((int)a, (int)b, c); }

// The scores of pages of one sequence and key-value head: kLanes lanes a page, 16 channels a lane. The CTA first
// makes the group's integers in shared memory, then its warps take pages in turn; heads by 8.
template <bool kBf16, int kLanes>
__global__ void __launch_bounds__(kWarps * 32) page_scores_kernel(const SelectParams p, int row_ctas) {
    constexpr int kGroups = 32 / kLanes;
    extern __shared__ __align__(16) uint8_t smem[];
    // per head kLanes * 16 bytes of its integers above zero, as many of those below; then a float 2^e a head
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int padded = (p.group + kHeads - 1) / kHeads * kHeads;
    uint4* const ints = reinterpret_cast<uint4*>(smem);  // [head][2][kLanes]
    float* const two = reinterpret_cast<float*>(smem + (size_t)padded * 2 * kLanes * 16);
    grid_begin();
    const int row = blockIdx.x / row_ctas, cta = blockIdx.x % row_ctas, b = row / p.hkv, hk = row % p.hkv;
    const int64_t room = p.per_seq * p.page_size;
    const int len = bounded_len(p.lens[b], room, p.status);
    const int pages = len ? (int)(((__umulhi(p.page_mul, (uint32_t)(len - 1)) + (uint64_t)(uint32_t)(len - 1)) >> p.page_shift) + 1) : 0;
    const int j_first = (cta * kWarps + warp) * kGroups, j_step = row_ctas * kWarps * kGroups;
    if (pages <= p.budget || cta * kWarps * kGroups >= pages) return;  // all are taken; nothing left for this CTA
    // ---- the queries' integers: kLanes lanes a head
    const int li = lane % kLanes, gr = lane / kLanes;
    for (int h0 = warp * kGroups; h0 < padded; h0 += kWarps * kGroups) {  // whole warps
        const int h = h0 + gr;
        float x[16];
        float a = 0.f;
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + b * p.q_batch + ((int64_t)hk * p.group + h) * p.q_head + 16 * li;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (h < p.group && 16 * li + 8 * k < p.d) w = *reinterpret_cast<const uint4*>(src + 8 * k);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = floats<kBf16>(ws[i]);
                x[8 * k + 2 * i] = f.x == f.x ? f.x : 0.f;
                x[8 * k + 2 * i + 1] = f.y == f.y ? f.y : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
        const int e = bound_exp(a);
        const float inv = exp2_of(-e);
        uint32_t up[4] = {}, down[4] = {};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int q = (int)fmaxf(fminf(rintf(x[i] * inv), 127.f), -127.f);
            up[i / 4] |= (uint32_t)max(q, 0) << (8 * (i % 4));
            down[i / 4] |= (uint32_t)(min(q, 0) & 0xff) << (8 * (i % 4));
        }
        if (h < padded) {
            ints[h * 2 * kLanes + li] = make_uint4(up[0], up[1], up[2], up[3]);
            ints[(h * 2 + 1) * kLanes + li] = make_uint4(down[0], down[1], down[2], down[3]);
            if (li == 0) two[h] = exp2_of(e);
        }
    }
    __syncthreads();
    const int32_t* table = p.table + b * p.table_stride;
    uint32_t* out = p.scores + (int64_t)row * p.per_seq;
    const bool whole = p.d % 16 == 0;
    for (int h0 = 0; h0 < padded; h0 += kHeads) {
        uint32_t up[kHeads][4], down[kHeads][4];
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            const uint4 u = ints[(h0 + h) * 2 * kLanes + li], d = ints[((h0 + h) * 2 + 1) * kLanes + li];
            up[h][0] = u.x, up[h][1] = u.y, up[h][2] = u.z, up[h][3] = u.w;
            down[h][0] = d.x, down[h][1] = d.y, down[h][2] = d.z, down[h][3] = d.w;
        }
        for (int64_t j0 = j_first; j0 < pages; j0 += j_step) {
            const int j = (int)j0 + gr;
            const int page = j < pages ? table[j] : -1;
            const bool good = (uint32_t)page < (uint64_t)p.num_pages && page >= 0;
            uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
            const int64_t at = (int64_t)page * p.hkv + hk;
            uint32_t byte = 0;
            if (good) {
                const int8_t* src = p.bounds + at * 2 * p.d + 16 * li;
                if (whole) {
                    if (16 * li < p.d) lo = *reinterpret_cast<const uint4*>(src), hi = *reinterpret_cast<const uint4*>(src + p.d);
                } else {
                    if (16 * li < p.d) {
                        const uint2 x = *reinterpret_cast<const uint2*>(src), y = *reinterpret_cast<const uint2*>(src + p.d);
                        lo.x = x.x, lo.y = x.y, hi.x = y.x, hi.y = y.y;
                    }
                    if (16 * li + 8 < p.d) {
                        const uint2 x = *reinterpret_cast<const uint2*>(src + 8), y = *reinterpret_cast<const uint2*>(src + p.d + 8);
                        lo.z = x.x, lo.w = x.y, hi.z = y.x, hi.w = y.y;
                    }
                }
                byte = p.bounds_exp[at];
            }
            float best = -INFINITY;
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                int u = 0;
                u = dot4(up[h][0], hi.x, dot4(up[h][1], hi.y, dot4(up[h][2], hi.z, dot4(up[h][3], hi.w, u))));
                u = dot4(down[h][0], lo.x, dot4(down[h][1], lo.y, dot4(down[h][2], lo.z, dot4(down[h][3], lo.w, u))));
#pragma unroll
                for (int off = kLanes / 2; off > 0; off >>= 1) u += __shfl_xor_sync(0xffffffffu, u, off);
                if (h0 + h < p.group) best = fmaxf(best, (float)u * two[h0 + h]);
            }
            if (j < pages && li == 0) {
                uint32_t key = good ? ordered(best * __uint_as_float(byte << 23)) : 0u;
                if (j < p.first || j >= pages - p.recent) key = kForced;
                out[j] = h0 == 0 ? key : max(out[j], key);
                if (!good && p.status) atomicOr(p.status, kStatusBadIndex);
            }
        }
    }
}

// ---------------------------------------------------------------------------- selection

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32, kHeld = 16;

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

// A CTA takes one sequence and head. Thread i has the scores of pages i per .. in registers, kHeld at most; more are read again.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
    __shared__ uint2 sums[kSelWarps];
    __shared__ uint32_t counts[2][kSelWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_begin();
    const int b = blockIdx.x / p.hkv;
    const int len = bounded_len(p.lens[b], p.per_seq * p.page_size, p.status);
    const int n = len ? (int)(((__umulhi(p.page_mul, (uint32_t)(len - 1)) + (uint64_t)(uint32_t)(len - 1)) >> p.page_shift) + 1) : 0;
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
    const int i0 = min((int)threadIdx.x * per, n), i1 = min(i0 + per, n);
    const bool held = per <= kHeld;
    uint32_t key[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) key[i] = held && i0 + i < i1 ? scores[i0 + i] : 0u;
    // ---- the largest x with at least `budget` keys >= x, bit by bit
    uint32_t least = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t x = least | (1u << bit);
        uint32_t mine = 0;
        if (held) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) mine += key[i] >= x;
        } else {
            for (int i = i0; i < i1; ++i) mine += scores[i] >= x;
        }
        mine = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) counts[bit & 1][warp] = mine;
        __syncthreads();
        uint32_t all = lane < kSelWarps ? counts[bit & 1][lane] : 0u;
        all = __reduce_add_sync(0xffffffffu, all);
        if (all >= (uint32_t)p.budget) least = x;
    }
    // ---- all above it, and the earliest of those equal to it
    uint2 mine = make_uint2(0, 0), total;
    auto each = [&](auto f) {
        if (held) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                if (i0 + i < i1) f(i0 + i, key[i]);
        } else {
            for (int i = i0; i < i1; ++i) f(i, scores[i]);
        }
    };
    each([&](int, uint32_t k) { mine.x += k > least, mine.y += k == least; });
    const uint2 before = scan2(mine, sums, &total);
    const uint32_t equal = (uint32_t)p.budget - total.x;  // taken of those equal
    uint32_t at = before.x + min(before.y, equal), seen = before.y;
    each([&](int i, uint32_t k) {
        if (k > least || (k == least && seen < equal)) {
            dst[at++] = table[i];
            if (i == n - 1) p.sel_lens[blockIdx.x] = p.budget * p.page_size - (int)((int64_t)n * p.page_size - len);
        } else if (i == n - 1) {
            p.sel_lens[blockIdx.x] = p.budget * p.page_size;
        }
        seen += k == least;
    });
}

template <bool kBf16, int kLanes>
cudaError_t launch_scores(const SelectParams& p, cudaStream_t stream) {
    const int padded = (p.group + kHeads - 1) / kHeads * kHeads;
    const size_t smem = (size_t)padded * (2 * kLanes * 16 + sizeof(float));
    // As many CTAs for a sequence and head as fill the SMs kResident times over, at most one for each kPages pages.
    constexpr int kPages = 64, kResident = 5;
    const int64_t rows = p.batch * p.hkv, most = (p.per_seq + kPages - 1) / kPages;
    const int64_t row_ctas = std::max<int64_t>(1, std::min(most, (152 * kResident + rows - 1) / rows));
    return launch_early(page_scores_kernel<kBf16, kLanes>, dim3((unsigned)(rows * row_ctas)), dim3(kWarps * 32), smem, stream, p, (int)row_ctas);
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
    const bool bf = p.dtype == kBf16;
    cudaError_t e = cudaSuccess;
    if (p.per_seq <= p.budget) {}  // every page is taken, without a look at the bounds
    else if (p.d <= 32) e = bf ? launch_scores<true, 2>(p, stream) : launch_scores<false, 2>(p, stream);
    else if (p.d <= 64) e = bf ? launch_scores<true, 4>(p, stream) : launch_scores<false, 4>(p, stream);
    else e = bf ? launch_scores<true, 8>(p, stream) : launch_scores<false, 8>(p, stream);
    if (e != cudaSuccess) return e;
    return launch_early(select_kernel, dim3((unsigned)(p.batch * p.hkv)), dim3(kSelThreads), 0, stream, p);
}

}  // namespace fa2
