// kv_select.cu - bounds of the keys in a page, and the pages whose keys can score highest for a query.
//
// Bounds: the lowest and the highest key of every channel, as 8-bit integers at a power of two of the page and
// head, rounded outwards: for 16 tokens of 128 channels in 16 bits 257 bytes for 8192 of keys and values. From 16-bit
// keys memory sets the pace (GB300, 9 prompts of up to 16384 tokens, 8 heads, 128 MB, 24 us, 5.3 TB/s); codes have to be
// widened and are compared two at a time, which does (60 of 100 cycles of the integer and comparison unit): e4m3, 66 MB,
// 18.7 us, 3.6 TB/s (24 when they were compared as bfloat16, by way of float32); 4 bits, 39 MB, 18.6 us. Half of a page's 910
// instructions find it and make its codes, as many as 32 rows of 128 take; larger pages have fewer, and for pages of a few keys
// that is the time (16 bits, pages of 8 39 us, of 1 265). The pages of a step of 33 sequences take 3.3 us: a launch and four reads one after another.
//
// Scores: sum_c max(q_c low_c, q_c high_c) is no less than q . k for any key within the bounds, with the query's 8-bit
// integers for q; for the query itself, which they round, it is an estimate that can lie below q . k. The integers, split
// into those above zero (which meet the highest keys) and those below (the lowest), make it a sum of integer products: exact, so that which pages are taken does not depend on the order of sums, and a
// float32 holds the result (below 2^21) times powers of two.
//
// Selection: the budget-th largest score by counting, the earlier page first among equals, pages in the order of
// their positions.
//
// Latency bounds it: each step of the chain length - table - bounds - scores - counts - pages waits 1 to 3 us, so it is one
// launch where it can be (with the attention, 16 sequences: 43.5 us, 48.8 in two). GB300, 128 of 1876 pages for each of 8
// heads of one sequence: 8.2 us; 64 of up to 2048 pages for each of 8 heads of 16 sequences, 42 MB of bounds: 21 us, 12 of
// them the scores of the longest row, whose tiles and queries pass through shared memory at half its rate.
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

// Lowest and highest of a lane's 16 channels over a page's rows, a group of kLanes lanes a row, kUnroll rows of each group at
// once. There is no other row or channel to skip: those behind the last one are the last one again.
template <int kForm, int kLanes>
struct PageKeys {
    static constexpr int kGroups = 32 / kLanes, kUnroll = kForm == kRows16 ? 4 : 8, kStep = kGroups * kUnroll;
    static constexpr int kWords = kForm == kRows16 ? 8 : (kForm == kRowsE4m3 ? 4 : 2);
    const PagedParams& c;
    const char *base, *second;  // of the lane's channels; 16-bit rows: of its last 8
    int64_t exp0;
    int live, gr, part;  // part: number of its 16 channels
    uint32_t k[kUnroll][kWords];
    uint32_t byte[kUnroll], scale[kUnroll];

    __device__ __forceinline__ void load(int s0) {  // rows s0 + gr, + kGroups, ...
#pragma unroll
        for (int n = 0; n < kUnroll; ++n) {
            if (s0 + n * kGroups >= live) continue;
            const int s = min(s0 + gr + n * kGroups, live - 1);
            const char* row = base + s * c.slot_stride;
            if constexpr (kForm == kRows16) {
                const uint4 x = *reinterpret_cast<const uint4*>(row), y = *reinterpret_cast<const uint4*>(second + s * c.slot_stride);
                k[n][0] = x.x, k[n][1] = x.y, k[n][2] = x.z, k[n][3] = x.w;
                k[n][4] = y.x, k[n][5] = y.y, k[n][6] = y.z, k[n][7] = y.w;
            } else if constexpr (kForm == kRowsE4m3) {
                const uint4 x = *reinterpret_cast<const uint4*>(row);
                k[n][0] = x.x, k[n][1] = x.y, k[n][2] = x.z, k[n][3] = x.w;
                byte[n] = c.k_exp[exp0 + s];
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(row);
                k[n][0] = x.x, k[n][1] = x.y;
                byte[n] = c.k_exp[exp0 + s];
                scale[n] = c.k_scale[(exp0 + s) * (c.d / 16) + part];
            }
        }
    }

    // The first rows are loaded. kHalf (codes): compared as halves at the power of two `top`; else as 16-bit floats that
    // hold every element. The groups then share the channels: from word w on, `words` pairs of each lane's 8, in l and u.
    template <bool kBf16, bool kHalf>
    __device__ __forceinline__ void compare(uint32_t top, int* w, float (&l)[kLanes == 8 ? 4 : 2], float (&u)[kLanes == 8 ? 4 : 2]) {
        constexpr bool kPairBf16 = !kHalf && (kBf16 || kForm != kRows16);
        using T = typename Pair<kPairBf16>::T;
        constexpr uint32_t kInf2 = kPairBf16 ? 0x7f807f80u : 0x7c007c00u;
        auto widen = [&](uint32_t word) { return *reinterpret_cast<T*>(&word); };
        auto bits = [&](T x) { return *reinterpret_cast<uint32_t*>(&x); };
        uint32_t lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[i] = kInf2, hi[i] = kInf2 | 0x80008000u;
        const uint32_t one = (15u - top) * 0x04000400u;  // 2^-top as two halves' bits, to which a byte adds
        for (int s0 = 0; s0 < live; s0 += kStep) {
            if (s0) load(s0);
#pragma unroll
            for (int n = 0; n < kUnroll; ++n) {
                if (s0 + n * kGroups >= live) continue;
                uint32_t x[8];
                if constexpr (kForm == kRows16) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = k[n][i];
                } else {
                    uint32_t s = 0;
                    if constexpr (kHalf) s = byte[n] * 0x04000400u + one;
                    if constexpr (kForm == kRowsE4m3) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) e4m3x4_to_f16x4(k[n][i], x[2 * i], x[2 * i + 1]);
                    } else {
                        uint32_t f[2][4];
                        e2m1x8_to_f16x8(k[n][0], f[0]);
                        e2m1x8_to_f16x8(k[n][1], f[1]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = f[i / 4][i % 4];
                        const uint32_t of16 = e4m3x2_to_f16x2(scale[n] * 0x101u);
                        s = kHalf ? hmul2(of16, s) : of16;
                    }
                    if constexpr (kHalf || kForm == kRowsE2m1) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = hmul2(x[i], s);
                    }
                    if constexpr (!kHalf) {
                        // (bfloat16 ends at 2^-133, a byte of 1 at 2^-136: any key below 2^-60 has bounds of -1, 0 or 1)
                        const float two = __uint_as_float(max(byte[n], 4u) << 23);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
                            x[i] = pack2<true>(y.x * two, y.y * two);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {  // (a NaN is not taken)
                    lo[i] = bits(__hmin2(widen(lo[i]), widen(x[i])));
                    hi[i] = bits(__hmax2(widen(hi[i]), widen(x[i])));
                }
            }
        }
        // two groups of lanes at a time join their words, each a half of them
        *w = 0;
#pragma unroll
        for (int off = kLanes, words = 8; off < 32; off <<= 1) {
            if (words > 1) words /= 2;
            const bool upper = (threadIdx.x & off) != 0;
            const bool halve = off < 8 * kLanes;
#pragma unroll
            for (int i = 0; i < words; ++i) {
                const uint32_t a = halve && upper ? lo[i + words] : lo[i], b = halve && upper ? hi[i + words] : hi[i];
                const uint32_t give_a = halve && !upper ? lo[i + words] : lo[i], give_b = halve && !upper ? hi[i + words] : hi[i];
                lo[i] = bits(__hmin2(widen(a), widen(__shfl_xor_sync(0xffffffffu, give_a, off))));
                hi[i] = bits(__hmax2(widen(b), widen(__shfl_xor_sync(0xffffffffu, give_b, off))));
            }
            if (halve && upper) *w += words;
        }
        const float power = kHalf ? __uint_as_float(top << 23) : 1.f;
#pragma unroll
        for (int i = 0; i < (kLanes == 8 ? 2 : 1); ++i) {
            const float2 x = floats<kPairBf16>(lo[i]), y = floats<kPairBf16>(hi[i]);
            l[2 * i] = x.x * power, l[2 * i + 1] = x.y * power, u[2 * i] = y.x * power, u[2 * i + 1] = y.y * power;
        }
    }

    // The largest finite magnitude in the lane's channels, which the lowest and the highest do not tell where they are infinite.
    // (Rare: a row at a time.)
    template <bool kBf16>
    __device__ __forceinline__ float largest() const {
        float a = 0.f;
#pragma unroll 1
        for (int s = gr; s < live; s += kGroups) {
            const float two = kForm == kRows16 ? 1.f : __uint_as_float((uint32_t)c.k_exp[exp0 + s] << 23);
            uint32_t of16 = 0;
            if constexpr (kForm == kRowsE2m1) of16 = e4m3x2_to_f16x2(c.k_scale[(exp0 + s) * (c.d / 16) + part] * 0x101u);
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {  // 8 channels
                const char* at = (kForm == kRows16 && i ? second : base + i * kWords / 2 * 4) + s * c.slot_stride;
                uint32_t x[4];
                if constexpr (kForm == kRows16) {
                    const uint4 w = *reinterpret_cast<const uint4*>(at);
                    x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
                } else if constexpr (kForm == kRowsE4m3) {
                    const uint2 w = *reinterpret_cast<const uint2*>(at);
                    e4m3x4_to_f16x4(w.x, x[0], x[1]);
                    e4m3x4_to_f16x4(w.y, x[2], x[3]);
                } else {
                    e2m1x8_to_f16x8(*reinterpret_cast<const uint32_t*>(at), x);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 y = floats<kForm == kRows16 && kBf16>(kForm == kRowsE2m1 ? hmul2(x[j], of16) : x[j]);
                    const float p = fabsf(y.x * two), q = fabsf(y.y * two);
                    a = fmaxf(a, fmaxf(p < INFINITY ? p : 0.f, q < INFINITY ? q : 0.f));
                }
            }
        }
        return a;
    }
};

// A warp takes one page of one sequence and one head: groups of kLanes lanes read slots in turn, 16 channels a lane.
template <bool kBf16, int kForm, int kLanes>
__global__ void __launch_bounds__(kWarps * 32) kv_bounds_kernel(const KvBoundsParams p) {
    const PagedParams& c = p.c;
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
        while (hi - lo > 1) {  // a lane a place
            const int apart = (hi - lo + 31) / 32, at = lo + lane * apart;
            const int before = __popc(__ballot_sync(0xffffffffu, at < hi && start(at < hi ? at : lo) <= w));
            lo += max(before - 1, 0) * apart;
            hi = min(lo + apart, hi);
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
    const int32_t page = c.table[b * c.table_stride + j];
    const Slot at = slot_of(c, page, 0);
    if (at.off < 0) return;
    const int live = (int)min((int64_t)c.page_size, len - j * c.page_size);
    const int li = lane % kLanes, gr = lane / kLanes;
    constexpr int kRowBits = kForm == kRows16 ? 16 : (kForm == kRowsE4m3 ? 8 : 4);
    const int pack = min(2 * li, c.d / 8 - 1), part = min(li, c.d / 16 - 1);  // (codes: whole 16)
    const char* row0 = c.k + at.off + h * c.head_stride;
    PageKeys<kForm, kLanes> keys{c, row0 + (kForm == kRows16 ? 16 * pack : 2 * kRowBits * part), row0 + 16 * min(2 * li + 1, c.d / 8 - 1),
                                 at.exp + (int64_t)h * c.page_size, live, gr, part};
    keys.load(0);
    constexpr int kOwn = kLanes == 8 ? 4 : 2;  // channels a lane ends with
    float l[kOwn], u[kOwn];
    int w0;
    if constexpr (kForm == kRows16) {
        keys.template compare<kBf16, false>(0, &w0, l, u);
    } else {
        // Below the largest byte of the page's rows by no more than 14, a row's codes (4 bits: times their scales), which are
        // multiples of 2^-9 (2^-10) of no more than 6 bits, are exact in half at the largest one's power.
        uint32_t top = 0, low = 255;
        for (int s = lane; s < live; s += 32) {
            const uint32_t x = c.k_exp[keys.exp0 + s];
            top = max(top, x);
            low = min(low, x);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        low = __reduce_min_sync(0xffffffffu, low);
        if (top - low <= 14) keys.template compare<true, true>(top, &w0, l, u);
        else keys.template compare<true, false>(top, &w0, l, u);
    }
    // ---- codes
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        if (l[i] > u[i]) l[i] = u[i] = 0.f;  // nothing but NaN
        a = fmaxf(a, fmaxf(fabsf(l[i]), fabsf(u[i])));
    }
    auto of_all = [](float x) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x))); };
    a = of_all(a);
    if (a == INFINITY) a = of_all(keys.template largest<kBf16>());
    const int e = bound_exp(a);
    const int channel = 16 * li + 2 * w0;
    if (channel >= c.d || gr >= 8) return;  // (16 groups end with the same twice)
    const float inv = exp2_of(-e);
    auto limited = [](float x) { return fmaxf(fminf(x, 127.f), -127.f); };  // (infinities)
    uint32_t low[kOwn], high[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {  // (the products round outwards too: a key far below the page's largest does not become 0)
        low[i] = (uint32_t)__float2int_rd(limited(__fmul_rd(l[i], inv)));
        high[i] = (uint32_t)__float2int_ru(limited(__fmul_ru(u[i], inv)));
    }
    uint32_t out[2] = {__byte_perm(low[0], low[1], 0x0040), __byte_perm(high[0], high[1], 0x0040)};
    if constexpr (kOwn == 4) {
        out[0] = __byte_perm(out[0], __byte_perm(low[2], low[3], 0x0040), 0x5410);
        out[1] = __byte_perm(out[1], __byte_perm(high[2], high[3], 0x0040), 0x5410);
    }
    const int64_t row = (int64_t)page * c.hkv + h;
    int8_t* dst = p.bounds + row * 2 * c.d + channel;
    if constexpr (kOwn == 4) {
        *reinterpret_cast<uint32_t*>(dst) = out[0];
        *reinterpret_cast<uint32_t*>(dst + c.d) = out[1];
    } else {
        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)out[0];
        *reinterpret_cast<uint16_t*>(dst + c.d) = (uint16_t)out[1];
    }
    if (lane == 0) p.bounds_exp[row] = (uint8_t)(e + 127);
}

template <bool kBf16, int kForm>
cudaError_t launch_bounds_form(const KvBoundsParams& p, cudaStream_t stream) {
    const int64_t pages = p.cu_new ? p.tokens / p.c.page_size + 2 * p.c.batch : p.c.batch;
    const dim3 grid((unsigned)((pages + kWarps - 1) / kWarps), (unsigned)p.c.hkv);
    if (p.c.d <= 32) return launch_early(kv_bounds_kernel<kBf16, kForm, 2>, grid, dim3(kWarps * 32), 0, stream, p);
    if (p.c.d <= 64) return launch_early(kv_bounds_kernel<kBf16, kForm, 4>, grid, dim3(kWarps * 32), 0, stream, p);
    return launch_early(kv_bounds_kernel<kBf16, kForm, 8>, grid, dim3(kWarps * 32), 0, stream, p);
}

// ---------------------------------------------------------------------------- scores

constexpr uint32_t kForced = 0xffffffffu;  // above every score's key; a page outside the cache: 0, below every score's
constexpr int kSelWarps = 8, kSelThreads = kSelWarps * 32, kSelPerSm = 2;
constexpr int kWideThreads = 1024;
constexpr int kBins = 1024;

// Unsigned numbers in the order of the floats (-0 as 0; NaN as -infinity: 0 times the power of a byte 255, infinity times
// that of a byte 0, whose bits would be those of kForced).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(fmaxf(x, -INFINITY) + 0.f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Pages that hold a length's keys.
__device__ __forceinline__ int pages_of(const SelectParams& p, int len) {
    if (len == 0) return 0;
    const uint32_t last = (uint32_t)len - 1;
    return (int)((__umulhi(p.page_mul, last) + last) >> p.page_shift) + 1;  // as page_of
}

// The query's side of the scores of one sequence and key-value head, in shared memory: a head's integers as halves,
// those below zero (which meet the lowest keys) and then those above, zeros behind 2 d; kPieces = ceil(d / 32).
template <int kPieces>
struct Queries {
    static constexpr int kRow = 128 * kPieces + 16;  // bytes a head, 8 rows in different banks
    static __host__ __device__ constexpr size_t bytes(int group) { return (size_t)((group + 7) / 8 * 8) * (kRow + sizeof(float2)); }
    uint8_t* rows;
    float2* stats;  // a head's -128 times the sum of its integers, and 2^e (0: no such head)
    __device__ Queries(uint8_t* smem, int padded) : rows(smem), stats(reinterpret_cast<float2*>(smem + (size_t)padded * kRow)) {}

    // A warp a head, 4 channels a lane (d <= 128).
    static __device__ __forceinline__ uint2 load(const SelectParams& p, int b, int hk, int h) {
        const int lane = threadIdx.x & 31;
        if (h >= p.group || 4 * lane >= p.d) return make_uint2(0, 0);
        return *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + b * p.q_batch + ((int64_t)hk * p.group + h) * p.q_head + 4 * lane);
    }
    // `first`: what load gave for this warp's first head. Every thread of the CTA calls it.
    template <bool kBf16>
    __device__ __forceinline__ void make(const SelectParams& p, int b, int hk, uint2 first) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, padded = (p.group + 7) / 8 * 8;
        for (int h = warp; h < padded; h += kSelWarps) {
            const uint2 w = h == warp ? first : load(p, b, hk, h);
            const float2 f = floats<kBf16>(w.x), g = floats<kBf16>(w.y);
            float x[4] = {f.x, f.y, g.x, g.y}, a = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (x[i] != x[i]) x[i] = 0.f;
                a = fmaxf(a, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
            const int e = bound_exp(a);
            const float inv = exp2_of(-e);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = fmaxf(fminf(rintf(x[i] * inv), 127.f), -127.f);
                sum += x[i];
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            uint2* dst = reinterpret_cast<uint2*>(rows + (size_t)h * kRow);  // 4 halves each
            if (4 * lane < p.d) {
                dst[lane] = make_uint2(pack2<false>(fminf(x[0], 0.f), fminf(x[1], 0.f)), pack2<false>(fminf(x[2], 0.f), fminf(x[3], 0.f)));
                dst[p.d / 4 + lane] = make_uint2(pack2<false>(fmaxf(x[0], 0.f), fmaxf(x[1], 0.f)), pack2<false>(fmaxf(x[2], 0.f), fmaxf(x[3], 0.f)));
            }
            for (int i = p.d / 2 + lane; i < 16 * kPieces; i += 32) dst[i] = make_uint2(0, 0);
            if (lane == 0) stats[h] = make_float2(-128.f * sum, h < p.group ? exp2_of(e) : 0.f);
        }
        __syncthreads();
    }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {  // else zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 load16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// Scores of pages tile * 16 .. of the sequence, tiles first, first + step, ...: put(page, key). The left operand's rows are
// the bounds of 16 pages, the right one's columns 8 heads' integers. Lane 4 g + t takes the 16-byte pieces t, t + 4, ...
// of the rows g and g + 8 (a product takes its terms in any order, both operands the same). A code plus 128, as a half's
// bits, is that many times 2^-24: two instructions for two codes, and the products' sums, of no more than 22 bits, are
// exact. (GB300, products a quarter of an SM can begin: one of 8-bit integers, 32 terms, every 63 cycles, one of halves,
// 16 terms, every 8; sums of four products 2 cycles for a 512th of either's 8192.)
// A page's number and its bounds follow one another from far away, 2 us and more: kDepth tiles are on their way or in
// use a warp; `meanwhile` runs while the first page numbers come. (In registers they would not fit, and a register that is spilled
// waits for its load: 35 us for 42 MB that way.)
constexpr int kDepth = 3;
template <int kPieces, typename Meanwhile, typename Put>
__device__ __forceinline__ void score_tiles(const SelectParams& p, const Queries<kPieces>& q, uint8_t* ring, const int32_t* table, int hk, int pages,
                                            int first, int step, Meanwhile meanwhile, Put put) {
    constexpr int kRow = 64 * kPieces, kFlip = kPieces % 2 == 0 ? 4 : 0;  // pieces of every other row change places: no bank twice
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t q_at = smem_u32(q.rows), my = smem_u32(ring) + (threadIdx.x >> 5) * (kDepth * 16 * kRow);
    const int per_row = p.d / 8;  // pieces
    const int8_t* const bounds = p.bounds + (int64_t)hk * 2 * p.d;
    const uint32_t page_bytes = (uint32_t)(p.hkv * 2 * p.d);
    auto look = [&](int64_t tile) { return lane < 16 && tile * 16 + lane < pages ? table[tile * 16 + lane] : -1; };
    // a tile's copies, one group of them; lane r has page r's power of two, or -1
    auto fetch = [&](int64_t tile, int page, uint32_t at) {
        float scale = -1.f;
        if (tile * 16 < pages) {
            const int good = page >= 0 && page < p.num_pages ? page : -1;
            if (good >= 0) scale = __uint_as_float((uint32_t)p.bounds_exp[(int64_t)good * p.hkv + hk] << 23);
#pragma unroll
            for (int i = 0; i < 2 * kPieces; ++i) {  // 32 pieces at a time, row by row
                const int n = 32 * i + lane, r = n / (4 * kPieces), piece = n % (4 * kPieces);
                const int here = __shfl_sync(0xffffffffu, good, r);
                const bool on = here >= 0 && piece < per_row;
                copy16(at + r * kRow + (piece ^ (r % 2 * kFlip)) * 16, bounds + (on ? (uint64_t)(uint32_t)here * page_bytes + 16 * piece : 0), on);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return scale;
    };
    auto finish = [&](int64_t tile, uint32_t at, float scale) {
        float best[2] = {-INFINITY, -INFINITY};
        for (int h0 = 0; h0 < p.group; h0 += 8) {
            float c2[2][4] = {};  // two chains of products
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const uint32_t b = q_at + (uint32_t)(h0 + g) * Queries<kPieces>::kRow + 128 * i + 32 * t;
                const uint4 b0 = load16(b), b1 = load16(b + 16);
                const uint32_t a = at + g * kRow + ((4 * i + t) ^ (g % 2 * kFlip)) * 16;  // (g + 8 is as odd as g)
                const uint4 u4 = load16(a), v4 = load16(a + 8 * kRow);
                const uint32_t bs[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
                const uint32_t u[4] = {u4.x, u4.y, u4.z, u4.w}, v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t y = u[w] ^ 0x80808080u, z = v[w] ^ 0x80808080u;
                    mma_f16(c2[w % 2], __byte_perm(y, 0, 0x4140), __byte_perm(z, 0, 0x4140), __byte_perm(y, 0, 0x4342), __byte_perm(z, 0, 0x4342), bs[2 * w],
                            bs[2 * w + 1]);
                }
            }
            const float c[4] = {c2[0][0] + c2[1][0], c2[0][1] + c2[1][1], c2[0][2] + c2[1][2], c2[0][3] + c2[1][3]};
#pragma unroll
            for (int n = 0; n < 2; ++n) {  // heads 2t, 2t+1
                if (h0 + 2 * t + n >= p.group) continue;
                const float2 s = q.stats[h0 + 2 * t + n];
                best[0] = fmaxf(best[0], fmaf(c[n], 0x1p24f, s.x) * s.y);
                best[1] = fmaxf(best[1], fmaf(c[2 + n], 0x1p24f, s.x) * s.y);
            }
        }
        // lane r has page r's score
        float score = 0.f;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float y = best[r];
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
            y = __shfl_sync(0xffffffffu, y, lane % 8 * 4);
            if (lane / 8 == r) score = y;
        }
        const int64_t j = tile * 16 + lane;
        if (lane < 16 && j < pages) {
            if (scale < 0.f && p.status) atomicOr(p.status, kStatusBadIndex);
            put((int)j, j < p.first || j >= pages - p.recent ? kForced : (scale >= 0.f ? ordered(score * scale) : 0u));
        }
    };
    int64_t tile = first;
    float scales[kDepth - 1];
    int ahead[kDepth];
#pragma unroll
    for (int i = 0; i < kDepth; ++i) ahead[i] = look(tile + i * (int64_t)step);
    meanwhile();
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) scales[i] = fetch(tile + i * (int64_t)step, ahead[i], my + i * 16 * kRow);
    int next = ahead[kDepth - 1];
    int use = 0, fill = kDepth - 1;
    for (; tile * 16 < pages; tile += step) {  // (no warp waits for another in here)
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
        __syncwarp();  // the tile is there for all lanes, and the one before is done with
        const float scale = scales[0];
#pragma unroll
        for (int i = 0; i + 1 < kDepth - 1; ++i) scales[i] = scales[i + 1];
        scales[kDepth - 2] = fetch(tile + (kDepth - 1) * (int64_t)step, next, my + fill * 16 * kRow);
        next = look(tile + kDepth * (int64_t)step);
        finish(tile, my + use * 16 * kRow, scale);
        use = use + 1 == kDepth ? 0 : use + 1;
        fill = fill + 1 == kDepth ? 0 : fill + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------------------- selection

// Sums over the CTA of a thread's two counts, packed as the halves of T, exclusive in thread order.
template <int kThreads, typename T>
__device__ __forceinline__ T scan(T v, T* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T upto = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T x = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += x;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    T before = 0;
    if constexpr (sizeof(T) == 4) {
        before = __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0);
    } else {
#pragma unroll 1  // (a kernel that runs once waits for its instructions: few of them)
        for (int w = 0; w < warp; ++w) before += sums[w];
    }
    return before + upto - v;
}

struct SelectSmem {
    unsigned long long sums[32];
    uint32_t bins[kBins];
    uint32_t found[3];
    uint32_t few;
    __align__(16) uint32_t list[32];
    __device__ __forceinline__ void begin() { found[0] = 0xffffffffu, found[1] = found[2] = few = 0; }
};

// The range of the scores that are not forced, and how many are.
struct Range {
    uint32_t lo = 0xffffffffu, hi = 0, forced = 0;
    __device__ __forceinline__ void add(uint32_t key) {
        if (key == kForced) ++forced;
        else lo = min(lo, key), hi = max(hi, key);
    }
    __device__ __forceinline__ void reduce() {  // over the warp
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        forced = __reduce_add_sync(0xffffffffu, forced);
    }
};

// All pages of row `row` (a sequence and head): there are no more than the budget.
__device__ __forceinline__ void take_all(const SelectParams& p, int row, const int32_t* table, int n, int len) {
    int32_t* dst = p.sel_table + (int64_t)row * p.budget;
    for (int i = threadIdx.x; i < p.budget; i += blockDim.x) {
        const int page = i < n ? table[i] : -1;
        dst[i] = page;
        if (i < n && (page < 0 || page >= p.num_pages) && p.status) atomicOr(p.status, kStatusBadIndex);
    }
    if (threadIdx.x == 0) p.sel_lens[row] = len;
}

// The budget of row `row` out of n > budget pages with keys key(0) .. key(n - 1). The budget-th largest is found by counting
// into kBins equal parts of the range that holds it, four times at the most (32 bits, 10 a time), mostly twice: the range
// begins as that of the scores there are.
// T: two counts of pages in one, 16 bits each (n < 2^16) or 32.
// kRanged: sm.found has the range and the number forced already, sm.few is 0.
template <int kThreads, typename T, bool kRanged, typename Key>
__device__ __forceinline__ void select_row(const SelectParams& p, SelectSmem& sm, int row, const int32_t* table, int n, int len, Key key) {
    constexpr int kHalf = 4 * sizeof(T);  // bits of a count
    constexpr T kOne = (T)1 << kHalf, kLow = kOne - 1;
    T* const sums = reinterpret_cast<T*>(sm.sums);
    const int lane = threadIdx.x & 31;
    // ---- the range of the scores that are not forced, and how many to take of those
    uint32_t lo, hi;
    if constexpr (!kRanged) {
        Range range;
#pragma unroll 1
        for (int i = threadIdx.x; i < n; i += kThreads) range.add(key(i));
        if (threadIdx.x == 0) sm.begin();
        range.reduce();
        __syncthreads();
        if (lane == 0) {
            atomicMin(&sm.found[0], range.lo);
            atomicMax(&sm.found[1], range.hi);
            if (range.forced) atomicAdd(&sm.found[2], range.forced);
        }
        __syncthreads();
    }
    lo = sm.found[0], hi = sm.found[1];
    uint32_t need = (uint32_t)p.budget - sm.found[2];
    uint32_t least = kForced - 1, equal = 0;  // all above `least` are taken and the earliest `equal` of those equal to it
#pragma unroll 1
    for (int round = 0; need && round < 4; ++round) {  // (four are enough)
        const int shift = max(0, 22 - __clz(hi - lo));  // (hi - lo) >> shift < kBins
        for (int i = threadIdx.x; i < kBins; i += kThreads) sm.bins[i] = 0;
        __syncthreads();  // (found is read)
#pragma unroll 1
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint32_t k = key(i);
            if (k >= lo && k <= hi) atomicAdd(&sm.bins[(k - lo) >> shift], 1u);
        }
        __syncthreads();
        // thread i has kPer parts from the top
        constexpr int kPer = kBins / kThreads;
        const int top = kBins - 1 - kPer * (int)threadIdx.x;
        uint32_t c[kPer], all = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) all += c[i] = sm.bins[top - i];
        uint32_t above = (uint32_t)scan<kThreads>((T)all, sums);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (above < need && need <= above + c[i]) sm.found[0] = top - i, sm.found[1] = above, sm.found[2] = c[i];
            above += c[i];
        }
        __syncthreads();
        lo += sm.found[0] << shift;
        hi = min(hi, lo + ((1u << shift) - 1));
        need -= sm.found[1];
        least = lo;
        if (shift == 0) {
            equal = need;
            break;
        }
        if (need == sm.found[2]) {  // the whole part: its lowest and all above
            equal = 0xffffffffu;
            break;
        }
        const uint32_t left = sm.found[2];
        if (left <= 32) {  // each warp ranks them
#pragma unroll 1
            for (int i = threadIdx.x; i < n; i += kThreads) {
                const uint32_t k = key(i);
                if (k >= lo && k <= hi) sm.list[atomicAdd(&sm.few, 1u)] = k;
            }
            __syncthreads();
            const uint32_t mine = lane < (int)left ? sm.list[lane] : 0u;
            uint32_t above_it = 0, alike = 0;
#pragma unroll 1
            for (uint32_t i = 0; i < left; i += 4) {
                const uint4 four = *reinterpret_cast<const uint4*>(&sm.list[i]);
                const uint32_t x[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) above_it += i + j < left && x[j] > mine, alike += i + j < left && x[j] == mine;
            }
            const uint32_t who = __ballot_sync(0xffffffffu, lane < (int)left && above_it < need && need <= above_it + alike);
            least = __shfl_sync(0xffffffffu, mine, __ffs(who) - 1);
            equal = need - __shfl_sync(0xffffffffu, above_it, __ffs(who) - 1);
            break;
        }
    }
    // ---- in the order of their positions: thread i has pages i per ..
    const int per = (n + kThreads - 1) / kThreads;
    const int i0 = (int)min((int64_t)threadIdx.x * per, (int64_t)n), i1 = min(i0 + per, n);
    T count = 0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = key(i);
        count += (k > least ? (T)1 : (T)0) + (k == least ? kOne : (T)0);
    }
    const T before = scan<kThreads>(count, sums);
    uint32_t seen = (uint32_t)(before >> kHalf), at = (uint32_t)(before & kLow) + min(seen, equal);
    // first the pages' places, then, side by side, what the table has there
    int32_t* dst = p.sel_table + (int64_t)row * p.budget;
    const bool listed = p.budget <= kBins;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = key(i);
        const bool take = k > least || (k == least && seen < equal);
        seen += k == least;
        if (take && at < (uint32_t)p.budget) {  // (as many as the budget, unless the table or the lengths changed meanwhile)
            if (listed) sm.bins[at++] = i;
            else dst[at++] = i;
        }
        if (i == n - 1) p.sel_lens[row] = p.budget * p.page_size - (take ? (int)((int64_t)n * p.page_size - len) : 0);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.budget; i += kThreads) dst[i] = table[listed ? (int)sm.bins[i] : dst[i]];
}

constexpr size_t ring_bytes(int pieces) { return (size_t)kSelWarps * kDepth * 16 * 64 * pieces; }

// The CTAs of a cluster of `ranks` share a sequence and head: all make scores, in the first one's shared memory, which selects.
template <bool kBf16, int kPieces>
__global__ void __launch_bounds__(kSelThreads, kSelPerSm) select_kernel(const SelectParams p, int ranks) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ SelectSmem sm;
    const int padded = (p.group + 7) / 8 * 8, row = blockIdx.x / ranks, rank = blockIdx.x % ranks, b = row / p.hkv, hk = row % p.hkv;
    Queries<kPieces> q(smem, padded);
    uint8_t* const ring = smem + Queries<kPieces>::bytes(p.group);
    uint32_t* scores = reinterpret_cast<uint32_t*>(ring + ring_bytes(kPieces));
    if (threadIdx.x == 0) sm.begin();
    cluster_arrive();  // all have started, the first one's counts are there: waited for before the first score
    grid_begin();
    const uint2 first_head = q.load(p, b, hk, threadIdx.x >> 5);
    const int len = bounded_len(p.lens[b], p.per_seq * p.page_size, p.status), n = pages_of(p, len);
    const int32_t* table = p.table + b * p.table_stride;
    if (n <= p.budget) {  // of the whole cluster
        cluster_wait();
        if (rank == 0) take_all(p, row, table, n, len);
        return;
    }
    const uint32_t to = cluster_map(smem_u32(scores), 0), found = cluster_map(smem_u32(sm.found), 0);
    Range range;
    score_tiles<kPieces>(
        p, q, ring, table, hk, n, rank * kSelWarps + (int)(threadIdx.x >> 5), ranks * kSelWarps,
        [&] {
            q.template make<kBf16>(p, b, hk, first_head);
            cluster_wait();
        },
        [&](int j, uint32_t key) {
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + 4 * j), "r"(key) : "memory");
            range.add(key);
        });
    range.reduce();
    if (threadIdx.x % 32 == 0) {
        asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(found), "r"(range.lo) : "memory");
        asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(found + 4), "r"(range.hi) : "memory");
        if (range.forced) asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(found + 8), "r"(range.forced) : "memory");
    }
    cluster_sync_all();
    if (rank == 0) select_row<kSelThreads, uint32_t, true>(p, sm, row, table, n, len, [&](int i) { return scores[i]; });
}

// The same for tables too wide for that, in two launches through the workspace.
template <bool kBf16, int kPieces>
__global__ void __launch_bounds__(kSelThreads, kSelPerSm) wide_scores_kernel(const SelectParams p, int row_ctas) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int padded = (p.group + 7) / 8 * 8, row = blockIdx.x / row_ctas, cta = blockIdx.x % row_ctas, b = row / p.hkv, hk = row % p.hkv;
    Queries<kPieces> q(smem, padded);
    grid_begin();
    const uint2 first_head = q.load(p, b, hk, threadIdx.x >> 5);
    const int n = pages_of(p, bounded_len(p.lens[b], p.per_seq * p.page_size, p.status));
    if (n <= p.budget || (int64_t)cta * kSelWarps * 16 >= n) return;
    uint32_t* out = p.scores + (int64_t)row * p.per_seq;
    score_tiles<kPieces>(
        p, q, smem + Queries<kPieces>::bytes(p.group), p.table + b * p.table_stride, hk, n, cta * kSelWarps + (int)(threadIdx.x >> 5), row_ctas * kSelWarps,
        [&] { q.template make<kBf16>(p, b, hk, first_head); }, [&](int j, uint32_t key) { out[j] = key; });
}
__global__ void __launch_bounds__(kWideThreads) wide_select_kernel(const SelectParams p) {
    __shared__ SelectSmem sm;
    const int row = blockIdx.x, b = row / p.hkv;
    grid_begin();
    const int len = bounded_len(p.lens[b], p.per_seq * p.page_size, p.status), n = pages_of(p, len);
    const int32_t* table = p.table + b * p.table_stride;
    if (n <= p.budget) return take_all(p, row, table, n, len);
    const uint32_t* scores = p.scores + (int64_t)row * p.per_seq;
    select_row<kWideThreads, unsigned long long, false>(p, sm, row, table, n, len, [&](int i) { return scores[i]; });
}
// Tables no wider than the budget: every page is taken, without a look at the bounds.
__global__ void __launch_bounds__(kSelThreads) take_all_kernel(const SelectParams p) {
    const int row = blockIdx.x, b = row / p.hkv;
    grid_begin();
    const int len = bounded_len(p.lens[b], p.per_seq * p.page_size, p.status);
    take_all(p, row, p.table + b * p.table_stride, pages_of(p, len), len);
}

template <bool kBf16, int kPieces>
cudaError_t launch_pieces(const SelectParams& p, cudaStream_t stream) {
    const int64_t rows = p.batch * p.hkv, tiles = (p.per_seq + 15) / 16, resident = 152 * kSelPerSm;
    const size_t q_bytes = Queries<kPieces>::bytes(p.group);  // 68 KB at most
    // One launch while a warp has no more than kRounds tiles (by the table's width: the lengths are on the device) and the
    // scores fit beside the queries.
    constexpr int kRounds = 8, kMostPages = 12 * 1024;
    const int64_t most = (tiles + kSelWarps - 1) / kSelWarps;
    const int ranks = (int)std::max<int64_t>(1, std::min<int64_t>({8, resident / rows, most}));
    const int slot = 208 + 4 * kBf16 + kPieces - 1;
    if (tiles <= (int64_t)ranks * kSelWarps * kRounds && p.per_seq <= kMostPages && rows * ranks <= INT32_MAX) {
        auto kern = select_kernel<kBf16, kPieces>;
        constexpr int kSmem = 217 * 1024;  // 68 + 96 + 48 KB at most
        cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), kSmem, slot);
        if (e != cudaSuccess) return e;
        const size_t smem = q_bytes + ring_bytes(kPieces) + (size_t)p.per_seq * sizeof(uint32_t);
        const int ask = ranks <= 2 ? ranks : (ranks <= 4 ? 4 : 8);
        if (ranks == 1 || cluster_fits(reinterpret_cast<const void*>(kern), kSelThreads, kSmem, ask, slot))
            return launch_early_cluster(kern, dim3((unsigned)(rows * ranks)), dim3(kSelThreads), smem, stream, (unsigned)ranks, p, ranks);
    }
    auto kern = wide_scores_kernel<kBf16, kPieces>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), 168 * 1024, slot + 8);
    if (e != cudaSuccess) return e;
    const int64_t row_ctas = std::max<int64_t>(1, std::min(most, resident / rows));
    e = launch_early(kern, dim3((unsigned)(rows * row_ctas)), dim3(kSelThreads), q_bytes + ring_bytes(kPieces), stream, p, (int)row_ctas);
    if (e != cudaSuccess) return e;
    return launch_early(wide_select_kernel, dim3((unsigned)rows), dim3(kWideThreads), 0, stream, p);
}

template <bool kBf16>
cudaError_t launch_select_type(const SelectParams& p, cudaStream_t stream) {
    switch ((p.d + 31) / 32) {
        case 1: return launch_pieces<kBf16, 1>(p, stream);
        case 2: return launch_pieces<kBf16, 2>(p, stream);
        case 3: return launch_pieces<kBf16, 3>(p, stream);
        default: return launch_pieces<kBf16, 4>(p, stream);
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
    if (p.per_seq <= p.budget) return launch_early(take_all_kernel, dim3((unsigned)(p.batch * p.hkv)), dim3(kSelThreads), 0, stream, p);
    return p.dtype == kBf16 ? launch_select_type<true>(p, stream) : launch_select_type<false>(p, stream);
}

}  // namespace fa2
