// kv_cache.cu - rows of keys and values into the pages of a cache, and back out.
//
// A row is one token's head_dim elements of one head, of K or of V. A warp takes one token (and
// a share of its heads): the page is looked up once for all its rows, then groups of lanes move
// one row each, 16 elements a lane to or from the 8-bit form and 8 a lane in the 16-bit form, so
// that every access to either side is a whole 16-byte vector.
//
// The 8-bit form: with a the row's largest finite magnitude, the scale is 2^e for the smallest
// e with a <= 448 2^e (448 the largest e4m3 value), from a's own exponent and fraction bits.
// A power of two makes x / 2^e exact, so a code depends on its rounding alone and reading back
// is exact in bfloat16. e >= -60 keeps 2^-e, 2^e and their products with sums inside float32.
//
// Bound by memory: each row is read once and written once. GB300: 563 MB (prompts into the 8-bit
// form, d = 64) in 86 us, 6.5 TB/s; 446 MB (8-bit rows read back, d = 128) in 75 us, 6.0 TB/s.
#include "paged.cuh"

namespace fa2 {
namespace {

constexpr int kWarps = 4;
constexpr int kMinExp = -60;
// Blocks from which a warp takes a whole token (with fewer, one round of its rows). GB300, 8 heads of
// d = 128, whole tokens against rounds: append e4m3 of 1200 tokens (300 blocks) 3.5 / 3.1 us, of 1800
// 3.8 / 4.6; 16 bits 3.2 / 3.7 and 3.5 / 5.1; 120,000 e4m3 111 / 178. (Reading e4m3 back, rounds stay
// ahead longer: 9600 tokens 16.1 / 13.2, 120,000 116 / 129.)
constexpr int kOneToken = 152 * 2;
// Blocks from which a warp takes kRows rounds of tokens of few heads, in 16 bits and in e4m3. One head,
// four rounds against one: e4m3 append d = 128 40,000 tokens (1250 blocks) 11.6 / 9.6 us, 160,000 29.4 /
// 29.9, 640,000 102 / 111; read 9.3 / 8.4, 23.4 / 24.7, 77 / 90. 16 bits d = 64 append 40,000 (1250)
// 7.4 / 6.7, 80,000 11.7 / 13.1, 640,000 61 / 84; read 20,000 3.2 / 3.2, 40,000 4.8 / 5.6, 640,000 50 / 82.
constexpr int kFewRounds16 = 152 * 8, kFewRoundsE4m3 = 152 * 32;

// e of the scale 2^e for a row whose largest finite magnitude is a.
__device__ __forceinline__ int scale_exp(float a) {
    if (a == 0.f) return 0;
    const uint32_t bits = __float_as_uint(a);
    const int k = (int)(bits >> 23) - 126;  // a = f 2^k, f in [1/2, 1) (a subnormal a reads as k = -126: clamped below)
    // 448 = 7/8 * 2^9: a <= 448 * 2^(k - 9) exactly when f <= 7/8
    const int e = k - 9 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < kMinExp ? kMinExp : e;
}

template <bool kBf16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
    if constexpr (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<__half2*>(&w));
}

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {  // nearest even; beyond 448: 448; NaN stays
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t to_e4m3x2_f16(uint32_t h2) {  // the same from two halves
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
    return r;
}

// The e4m3 codes of a lane's 16 elements, and e of their row's scale 2^e. Every lane of the warp calls
// it; kLanes lanes hold a row. The magnitudes of 16-bit floats are ordered as their bits are, so the
// largest one is found two at a time on the bits; rows with an infinity or a NaN (rare) take a second
// look that leaves those out.
template <bool kBf16, int kLanes>
__device__ __forceinline__ uint4 quantise(const uint32_t (&w)[8], int* exp) {
    constexpr uint32_t kInf = kBf16 ? 0x7f80u : 0x7c00u;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = __vmaxu2(m, w[j] & 0x7fff7fffu);
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
    m = max(m & 0xffffu, m >> 16);
    if (__any_sync(0xffffffffu, m >= kInf)) {
        m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
            m = max(m, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
        }
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
    }
    const float a = kBf16 ? __uint_as_float(m << 16) : __half2float(__ushort_as_half((unsigned short)m));
    const int e = scale_exp(a);
    *exp = e;
    uint32_t o[4];
    if (!kBf16 && !__any_sync(0xffffffffu, e < -15)) {
        // 2^-e (e <= 8) is a normal half: the products are exact down to 2^-24, far below a code's
        // smallest half step 2^-10
        const __half2 inv = __half2half2(__ushort_as_half((unsigned short)((15 - e) << 10)));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&w[j]), inv);
            const uint32_t c = to_e4m3x2_f16(*reinterpret_cast<const uint32_t*>(&x));
            o[j >> 1] = (j & 1) ? o[j >> 1] | (c << 16) : c;
        }
    } else {
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e, e in [-60, 120]
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = widen2<kBf16>(w[j]);
            const uint32_t c = to_e4m3x2(f.x * inv, f.y * inv);
            o[j >> 1] = (j & 1) ? o[j >> 1] | (c << 16) : c;
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The cache side of one token: bytes / scale bytes, head 0.
struct Token {
    int64_t cache_off, exp_off;
};

// Where row t of k and v, or position t of sequence b_read, lies; false: nowhere.
__device__ __forceinline__ bool find_token(const KvRowsParams& p, int64_t t, int b_read, Token* out) {
    const PagedParams& c = p.c;
    int64_t pos;
    int b;
    if (p.read) {
        b = b_read;
        pos = t;
        if (pos >= bounded_len(c.lens[b], c.room, c.status)) return false;
    } else {
        int first = (int)t, end = (int)t + 1;
        if (p.cu_new) {
            // the last sequence that begins at or before row t
            int lo = 0, hi = (int)c.batch;  // cu_new[lo] <= t < cu_new[hi], were it ascending
            if (t < p.cu_new[0] || t >= p.cu_new[hi]) return false;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (p.cu_new[mid] <= t) lo = mid;
                else hi = mid;
            }
            b = lo;
            first = p.cu_new[b];
            end = p.cu_new[b + 1];
        } else {
            b = (int)t;
            if (c.lens[b] == 0) return false;
        }
        pos = (int64_t)c.lens[b] - end + t;
        if (t < first || t >= end || pos < 0 || pos >= c.room) {
            if (c.status) atomicOr(c.status, kStatusBadIndex);
            return false;
        }
    }
    const int at = page_of(c, (int)pos);
    const Slot s = slot_of(c, c.table[b * c.table_stride + at], (int)pos - at * c.page_size);
    if (s.off < 0) return false;
    out->cache_off = s.off;
    out->exp_off = s.exp;
    return true;
}

// Moves kRows rows a lane, all loads first: there(i) says whether the i-th exists, the others give its
// addresses (cache side, tensor side, scale byte). Every lane of the warp calls it: the kLanes lanes
// of a row find its largest magnitude together.
template <bool kBf16, bool kE4m3, bool kRead, int kLanes, int kRows, typename There, typename Cache, typename Tensor, typename Exp>
__device__ __forceinline__ void move_rows(int li, There there, Cache cache_ptr, Tensor row_ptr, Exp exp_ptr) {
    uint4 in[kRows][kE4m3 ? 2 : 1];
    int byte[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        in[i][0] = make_uint4(0, 0, 0, 0);
        if constexpr (kE4m3) in[i][1] = make_uint4(0, 0, 0, 0);
        byte[i] = 127;
        if (!there(i)) continue;
        if constexpr (kRead) {
            in[i][0] = *reinterpret_cast<const uint4*>(cache_ptr(i));
            if constexpr (kE4m3) byte[i] = *exp_ptr(i);
        } else {
            const uint4* src = reinterpret_cast<const uint4*>(row_ptr(i));
            in[i][0] = src[0];
            if constexpr (kE4m3) in[i][1] = src[1];
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if constexpr (!kE4m3) {
            if (there(i)) *reinterpret_cast<uint4*>(kRead ? row_ptr(i) : cache_ptr(i)) = in[i][0];
        } else if constexpr (kRead) {
            if (there(i)) {
                const uint32_t w[4] = {in[i][0].x, in[i][0].y, in[i][0].z, in[i][0].w};
                const float scale = __uint_as_float((uint32_t)byte[i] << 23);
                uint32_t o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t h2[2];
                    e4m3x4_to_f16x4(w[j], h2[0], h2[1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2[e]));
                        o[2 * j + e] = pack2<kBf16>(f.x * scale, f.y * scale);
                    }
                }
                uint4* dst = reinterpret_cast<uint4*>(row_ptr(i));
                dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
                dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
        } else {
            const uint32_t w[8] = {in[i][0].x, in[i][0].y, in[i][0].z, in[i][0].w,
                                   in[i][1].x, in[i][1].y, in[i][1].z, in[i][1].w};
            int e;
            const uint4 codes = quantise<kBf16, kLanes>(w, &e);
            if (there(i)) {
                *reinterpret_cast<uint4*>(cache_ptr(i)) = codes;
                if (li == 0) *exp_ptr(i) = (uint8_t)(e + 127);
            }
        }
    }
}

// A warp moves kTok tokens one after another, looked up at once, a lane for each; kLanes lanes move
// a row, of each token's 2 hkv rows (heads of K, then of V) rows r0, r0 + 32 / kLanes, ..., kRows of
// them at a time.
template <bool kBf16, bool kE4m3, bool kRead, int kLanes, int kRows, int kTok>
__global__ void __launch_bounds__(kWarps * 32) kv_rows_kernel(const KvRowsParams p, int rows_per_warp) {
    const PagedParams& c = p.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * kTok;
    grid_begin();
    if (t0 >= p.tokens) return;
    Token found{-1, -1};
    {
        const int64_t t = t0 + lane % kTok;
        if (t < p.tokens && !find_token(p, t, blockIdx.z, &found)) found.cache_off = -1;
    }
    constexpr int kGroups = 32 / kLanes;
    constexpr int kElems = kE4m3 ? 16 : 8;  // elements a lane
    const int li = lane % kLanes;
    const bool on = li * kElems < c.d;
    const int total = 2 * c.hkv;
    const int begin = blockIdx.y * rows_per_warp, stop = min(total, begin + rows_per_warp);
    const int64_t k_step = p.read ? p.ks[2] : p.ks[0], v_step = p.read ? p.vs[2] : p.vs[0];
    const int64_t k_base = p.read ? blockIdx.z * p.ks[0] : 0, v_base = p.read ? blockIdx.z * p.vs[0] : 0;
    for (int n = 0; n < kTok; ++n) {
        const Token tok{__shfl_sync(0xffffffffu, found.cache_off, n), kE4m3 ? __shfl_sync(0xffffffffu, found.exp_off, n) : 0};
        if (tok.cache_off < 0) continue;
        const int64_t k_off = k_base + (t0 + n) * k_step, v_off = v_base + (t0 + n) * v_step;
        for (int r0 = begin + lane / kLanes; r0 - lane / kLanes < stop; r0 += kGroups * kRows) {
            auto head = [&](int i, bool* v) {
                const int r = r0 + i * kGroups;
                *v = r >= c.hkv;
                return *v ? r - c.hkv : r;
            };
            move_rows<kBf16, kE4m3, kRead, kLanes, kRows>(
                li, [&](int i) { return r0 + i * kGroups < stop && on; },
                [&](int i) {
                    bool v;
                    const int h = head(i, &v);
                    return (v ? c.v : c.k) + tok.cache_off + h * c.head_stride + li * 16;
                },
                [&](int i) {
                    bool v;
                    const int h = head(i, &v);
                    return (v ? p.v + v_off + h * p.vs[1] : p.k + k_off + h * p.ks[1]) + li * kElems * 2;
                },
                [&](int i) {
                    bool v;
                    const int h = head(i, &v);
                    return (v ? c.v_exp : c.k_exp) + tok.exp_off + (int64_t)h * c.page_size;
                });
        }
    }
}

// Few heads: tokens whose rows fill no more than half of a warp's groups of lanes. The group's row is
// group % (1 << shift) of the token group >> shift further on; kRows rounds of tokens.
template <bool kBf16, bool kE4m3, bool kRead, int kLanes, int kRows>
__global__ void __launch_bounds__(kWarps * 32) kv_few_heads_kernel(const KvRowsParams p, int shift) {
    const PagedParams& c = p.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kGroups = 32 / kLanes;
    const int li = lane % kLanes, group = lane / kLanes, r = group & ((1 << shift) - 1), step = kGroups >> shift;
    const int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * kRows * step + (group >> shift);
    grid_begin();
    const bool on = li * (kE4m3 ? 16 : 8) < c.d && r < 2 * c.hkv, v = r >= c.hkv;
    const int h = v ? r - c.hkv : r;
    Token tok[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t t = t0 + i * step;
        tok[i].cache_off = -1;
        if (on && t < p.tokens && !find_token(p, t, blockIdx.z, &tok[i])) tok[i].cache_off = -1;
    }
    char* const cache = (v ? c.v : c.k) + h * c.head_stride + li * 16;
    char* const rows = (v ? p.v + h * p.vs[1] : p.k + h * p.ks[1]) + li * (kE4m3 ? 32 : 16) +
                       (p.read ? blockIdx.z * (v ? p.vs[0] : p.ks[0]) : 0);
    const int64_t row_step = p.read ? (v ? p.vs[2] : p.ks[2]) : (v ? p.vs[0] : p.ks[0]);
    move_rows<kBf16, kE4m3, kRead, kLanes, kRows>(
        li, [&](int i) { return tok[i].cache_off >= 0; }, [&](int i) { return cache + tok[i].cache_off; },
        [&](int i) { return rows + (t0 + i * step) * row_step; },
        [&](int i) { return (v ? c.v_exp : c.k_exp) + tok[i].exp_off + (int64_t)h * c.page_size; });
}

template <bool kBf16, bool kE4m3, bool kRead, int kLanes>
cudaError_t launch_lanes(const KvRowsParams& p, cudaStream_t stream) {
    constexpr int kGroups = 32 / kLanes, kRows = 4, kTok = 2;
    const int total = 2 * p.c.hkv;
    const unsigned batch = (unsigned)(p.read ? p.c.batch : 1);
    int shift = 0;  // 1 << shift groups of lanes for a token's rows
    while ((1 << shift) < total) ++shift;
    if ((2 << shift) <= kGroups) {
        const int64_t per = (int64_t)kWarps * kRows * (kGroups >> shift);
        if ((p.tokens + per - 1) / per * batch >= (kE4m3 ? kFewRoundsE4m3 : kFewRounds16)) {
            const dim3 grid((unsigned)((p.tokens + per - 1) / per), 1, batch);
            return launch_early(kv_few_heads_kernel<kBf16, kE4m3, kRead, kLanes, kRows>, grid, dim3(kWarps * 32), 0, stream, p, shift);
        }
        const int64_t one = (int64_t)kWarps * (kGroups >> shift);
        const dim3 grid((unsigned)((p.tokens + one - 1) / one), 1, batch);
        return launch_early(kv_few_heads_kernel<kBf16, kE4m3, kRead, kLanes, 1>, grid, dim3(kWarps * 32), 0, stream, p, shift);
    }
    auto blocks = [&](int tok) { return (p.tokens + kWarps * tok - 1) / (kWarps * tok); };
    // A warp takes kTok whole tokens while that gives every SM several blocks, one token with fewer,
    // and with few tokens one round of a token's rows. 120,000 tokens, 8 heads, d = 128, append e4m3 /
    // 16 bits / read e4m3: kTok 1 118.6 / 144.6 / 126.4 us, 2 111.1 / 145.5 / 116.3, 4 113.2 / 148.7 /
    // 118.6; kRows 2 113.0 / 146.8 / 115.0, 8 171.5 / 144.6 / 130.8.
    if (blocks(kTok) * batch >= 152 * 8) {
        const dim3 grid((unsigned)blocks(kTok), 1, batch);
        return launch_early(kv_rows_kernel<kBf16, kE4m3, kRead, kLanes, kRows, kTok>, grid, dim3(kWarps * 32), 0, stream, p, total);
    }
    if (blocks(1) * batch >= kOneToken) {
        const dim3 grid((unsigned)blocks(1), 1, batch);
        return launch_early(kv_rows_kernel<kBf16, kE4m3, kRead, kLanes, kRows, 1>, grid, dim3(kWarps * 32), 0, stream, p, total);
    }
    const dim3 grid((unsigned)blocks(1), (unsigned)((total + kGroups - 1) / kGroups), batch);
    return launch_early(kv_rows_kernel<kBf16, kE4m3, kRead, kLanes, 1, 1>, grid, dim3(kWarps * 32), 0, stream, p, kGroups);
}

template <bool kBf16, bool kE4m3, bool kRead>
cudaError_t launch_type(const KvRowsParams& p, cudaStream_t stream) {
    const int lanes = kE4m3 ? (p.c.d + 15) / 16 : (p.c.d + 7) / 8;
    if (lanes <= 2) return launch_lanes<kBf16, kE4m3, kRead, 2>(p, stream);
    if (lanes <= 4) return launch_lanes<kBf16, kE4m3, kRead, 4>(p, stream);
    if (lanes <= 8) return launch_lanes<kBf16, kE4m3, kRead, 8>(p, stream);
    return launch_lanes<kBf16, kE4m3, kRead, 16>(p, stream);
}

}  // namespace

cudaError_t launch_kv_rows(const KvRowsParams& p, cudaStream_t stream) {
    const bool bf = p.c.dtype == kBf16;
    if (!p.c.e4m3)  // words are moved without a look at them
        return p.read ? launch_type<true, false, true>(p, stream) : launch_type<true, false, false>(p, stream);
    if (p.read) return bf ? launch_type<true, true, true>(p, stream) : launch_type<false, true, true>(p, stream);
    return bf ? launch_type<true, true, false>(p, stream) : launch_type<false, true, false>(p, stream);
}

}  // namespace fa2
