// kv_rope.cuh - new tokens' queries and keys turned by their positions, and their keys and values into the
// pages of a cache, in one pass; fa2_kv_append's 4-bit rows (nothing turned).
//
// As two calls (fa2_rope, fa2_kv_append) the keys are written and read once more than needed and every step
// pays two launches. Here each row is read once and written once: bytes set the pace of prompts, the chain
// length - page - row - store that of a step. GB300: 16-bit prompts (6 of up to 6100, 32 and 8 heads of 128, 334 MB)
// 57.8 us, 5.8 TB/s; into e4m3 (11 of up to 16384, 16 and 16 heads of 64, half of each turned, 937 MB) 163 us, 5.7 TB/s:
// memory, as far as the rounds on their way reach. Into 4 bits (9 of up to 16384, 8 heads of 128, 319 MB) 94 us, 3.4 TB/s,
// keys turned on the way 120 (interleaved pairs 110): maxima, quotients and conversions. A step of 33 sequences into e4m3 4.4 us.
//
// A warp takes a token (and a share of its rows); kLanes lanes hold a row, 16 elements each, as two packs of 8:
// i .. i + 7 and i + rot / 2 .. in the half layout, any two in the interleaved one, so that every pair lies in one
// lane whichever the layout, accesses are whole 16-byte vectors, and the 8 sines and cosines a lane needs are
// the same for all rows of the token (rope.cuh makes them from the position in fixed point). Hence rot a multiple of 16: whole
// packs turn with whole packs. (fa2_rope, which has narrower accesses, takes any even one.)
//
// The 8- and 4-bit forms take a row's power of two from the row as it came (the magnitudes of 16-bit floats are
// ordered as their bits are): a rotation by any angle makes an element no more than sqrt(2) |magnitude| times the
// largest, so one bit more, and as many as the magnitude has, are always enough, and what the 8-bit floats lose
// by it lies at the bottom of their range. It does not depend on how sines round.
//
// The 4-bit form: x 2^-e < 2^10 (turned: 2^10 sqrt(2) < 448 * 6), 16 elements' scale is max / 6 as an 8-bit float,
// codes are x 2^-e / scale, the scales' reciprocals a table. Both quotients are rounded exactly: with r = 1 / s to
// nearest, q = x r, the remainder x - q s is exact in one fused step and q + r (x - q s) is x / s to nearest (P. W.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34,
// 1990), which keeps every tie between two codes a tie.
#pragma once

#include <algorithm>

#include "paged.cuh"
#include "rope.cuh"

namespace fa2 {
namespace {

constexpr int kWarps = 4;
// CTAs an SM: 96 registers a thread, room for the rounds on their way (launch_lanes). With pairs in halves and two rounds ahead
// 4-bit rows spill 16 to 24 bytes, with three ahead e4m3 rows of up to 64 spill 16.
constexpr int kPerSm = 5;
constexpr int kMinExp = -60, kMaxExp = 120;

template <bool kBf16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
    if constexpr (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<__half2*>(&w));
}

// Two float32 products, or fused products and sums, in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\tfma.rn.f32x2 z, x, y, w;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// The larger magnitudes of the even and of the odd elements of 8 16-bit floats: their bits are ordered as they are.
__device__ __forceinline__ uint32_t pack_max(const uint4& w) {
    const uint32_t k = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k));
}
template <bool kBf16>
__device__ __forceinline__ float magnitude_of(uint32_t bits) {
    return kBf16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half((unsigned short)bits));
}

// The largest finite magnitude of a row, a lane's 16 elements in `in`, `m` their pack_max; kLanes lanes hold the row, every lane
// of the warp calls it.
template <bool kBf16, int kLanes>
__device__ __forceinline__ float row_max(const uint4 (&in)[2], uint32_t m) {
    constexpr uint32_t kInf = kBf16 ? 0x7f80u : 0x7c00u;
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
    m = max(m & 0xffffu, m >> 16);
    if (__any_sync(0xffffffffu, m >= kInf)) {  // rare: look again without infinities and NaN
        const uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
        m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
            m = max(m, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
        }
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
    }
    return magnitude_of<kBf16>(m);
}

// e of a row's power of two 2^e for its largest magnitude a before any rotation, `more` for what that can add.
template <int kForm>
__device__ __forceinline__ int row_exp(float a, int more) {
    int e = 0;
    if (a > 0.f) {
        const uint32_t bits = __float_as_uint(a);
        const int k = (int)(bits >> 23) - 126;  // a = f 2^k, f in [1/2, 1) (a subnormal a: k = -126, and the limit below)
        e = kForm == kRowsE2m1 ? k - 10 : k - 9 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);  // e4m3: a <= 448 2^e
        e = max(e, kMinExp);
    }
    return min(e + more, kMaxExp);
}
__device__ __forceinline__ float exp2_of(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {  // nearest even; beyond 448: 448; NaN stays
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight e2m1 codes, nearest even, beyond 6: 6.
__device__ __forceinline__ uint32_t to_e2m1x8(const float2 (&x)[4]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r) : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y));
    return r;
}

// x / s to nearest, for finite x and s with r = 1 / s to nearest
__device__ __forceinline__ float divide(float x, float s, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, s, x), r, q);
}

// The largest of 8 magnitudes, as bits: NaN above infinity above the finite ones.
__device__ __forceinline__ uint32_t max_bits(const float2 (&x)[4]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(__float_as_uint(x[i].x) & 0x7fffffffu, __float_as_uint(x[i].y) & 0x7fffffffu));
    return m;
}

// The scale byte of 16 elements whose largest magnitude has these bits, at a row's power of two 2^-e = inv.
__device__ __forceinline__ uint32_t group_scale(uint32_t bits, float inv) {
    if (bits > 0x7f800000u) return 0x7fu;   // a NaN
    if (bits == 0x7f800000u) return 0x7eu;  // an infinity: 448
    return to_e4m3x2(divide(__uint_as_float(bits) * inv, 6.f, 1.f / 6.f), 0.f) & 0xffu;
}

// The codes of 8 elements at a scale byte of group_scale and a row's power of two; `reciprocal[i]`: what scale byte i stands for, and
// 1 over that (0 for 0). The powers of two go with the scale: x / (s 2^e), exactly x 2^-e / s.
__device__ __forceinline__ uint32_t group_codes(const float2 (&x)[4], uint32_t scale, float two, float inv, const float2* reciprocal) {
    const float2 f = reciprocal[scale];
    const float s = f.x * two, r = f.y * inv;
    float2 y[4];
    if (scale < 0x7eu) {
        const float2 r2 = make_float2(r, r), s2 = make_float2(-s, -s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // divide, two at a time
            const float2 q = mul2(x[i], r2);
            y[i] = fma2(fma2(q, s2, x[i]), r2, q);
        }
    } else {  // an infinity's remainder is none
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = make_float2(__fdiv_rn(x[i].x * inv, f.x), __fdiv_rn(x[i].y * inv, f.x));
    }
    return to_e2m1x8(y);
}

// Where a token lies: bytes / scale bytes of the cache, head 0 (-1: its page is outside); its position (-1: none).
struct Spot {
    int64_t cache_off, exp_off;
    int pos;
};

// Warp w takes tokens w, w + all warps, ..., looked up 32 at once, a lane for each. It has kAhead rounds of rows (one for
// each group of lanes) on their way while it works on one.
template <bool kBf16, int kForm, bool kInterleaved, int kLanes, int kAhead>
__global__ void __launch_bounds__(kWarps * 32, kPerSm) rope_append_kernel(const RopeAppendParams p, int slots_per_warp) {
    const PagedParams& c = p.rows.c;
    constexpr int kGroups = 32 / kLanes;
    __shared__ uint64_t turns[64];
    __shared__ float2 reciprocal[kForm == kRowsE2m1 ? 128 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * kWarps + warp, step = (int64_t)gridDim.x * kWarps;
    if constexpr (kForm == kRowsE2m1) {
        const float s = __half2float(__ushort_as_half((unsigned short)e4m3x2_to_f16x2(threadIdx.x & 127)));
        reciprocal[threadIdx.x & 127] = make_float2(s, s > 0.f ? __frcp_rn(s) : 0.f);
    }
    grid_begin();
    if (p.rot)
        for (int i = threadIdx.x; i < p.rot / 2; i += kWarps * 32) turns[i] = turns_of(p.inv_freq[i]);
    __syncthreads();
    if (t0 >= p.rows.tokens) return;
    const int tokens = (int)((p.rows.tokens - t0 + step - 1) / step);  // of this warp
    Spot found{-1, -1, -1};
    auto look = [&](int n) {  // lane l: the warp's token n + l
        found = Spot{-1, -1, -1};
        int b;
        int64_t pos;
        if (n + lane < tokens && place_of_row(c, p.rows.cu_new, t0 + (n + lane) * step, &b, &pos)) {
            found.pos = (int)pos;
            const int at = page_of(c, found.pos);
            const Slot s = slot_of(c, c.table[b * c.table_stride + at], found.pos - at * c.page_size);
            found.cache_off = s.off;
            found.exp_off = s.exp;
        }
    };
    const int li = lane % kLanes, gr = lane / kLanes;
    // the lane's packs and whether they turn
    int i0, i1;
    bool on0, on1, turned0, turned1;
    if (!kInterleaved && 16 * li < p.rot) {  // elements that turn with one another
        i0 = 8 * li, i1 = p.rot / 2 + 8 * li;
        on0 = on1 = turned0 = turned1 = true;
    } else if (kForm == kRowsE2m1) {  // 16 in a row, one scale
        i0 = 16 * li, i1 = i0 + 8;
        on0 = i0 < c.d, on1 = i1 < c.d;
        turned0 = turned1 = i0 < p.rot;
    } else {  // as far apart as the lanes: a row's packs of either number are one after another in memory
        const int from = kInterleaved ? 0 : p.rot, m = li - from / 16, apart = (c.d - from + 15) / 16;
        i0 = from + 8 * m, i1 = i0 + 8 * apart;
        on0 = m < apart, on1 = on0 && i1 < c.d;
        turned0 = i0 < p.rot, turned1 = i1 < p.rot;  // (whole packs)
    }
    // 4 bits: the lane and the pack that hold the other 8 of the 16 elements around each pack
    const bool apart = !kInterleaved && p.rot;  // (else the lane itself)
    auto holder = [&](int pack, int* second) {  // of elements 8 pack ..
        const int k = apart ? p.rot / 16 : 0;
        const bool half = pack < 2 * k;
        *second = half ? pack >= k : pack & 1;
        return lane - li + (half ? (pack < k ? pack : pack - k) : pack / 2);
    };
    int second0 = 0, second1 = 0, from0 = 0, from1 = 0;
    if constexpr (kForm == kRowsE2m1) {
        from0 = holder((i0 / 8) ^ 1, &second0) & 31;
        from1 = holder((i1 / 8) ^ 1, &second1) & 31;
    }
    // rows: the queries', from a whole round on the keys', the values'
    const int q_slots = (p.heads + kGroups - 1) / kGroups * kGroups, total = q_slots + 2 * c.hkv;
    const int begin = blockIdx.y * slots_per_warp, stop = min(total, begin + slots_per_warp);

    // ---- rounds of rows on their way: token fetch_n, rows fetch_s + gr
    int fetch_n = 0, fetch_s = begin;
    auto fetch = [&](uint4 (&in)[2]) {
        in[0] = in[1] = make_uint4(0, 0, 0, 0);
        const int64_t t = t0 + fetch_n * step;
        const int r = fetch_s + gr, k = r - q_slots;
        if (fetch_n < tokens && r < stop) {
            const char* src = nullptr;
            if (fetch_s < q_slots) {
                if (r < p.heads) src = p.q + t * p.qs[0] + r * p.qs[1];
            } else {
                src = k >= c.hkv ? p.rows.v + t * p.rows.vs[0] + (k - c.hkv) * p.rows.vs[1] : p.rows.k + t * p.rows.ks[0] + k * p.rows.ks[1];
            }
            if (src && on0) in[0] = *reinterpret_cast<const uint4*>(src + 2 * i0);
            if (src && on1) in[1] = *reinterpret_cast<const uint4*>(src + 2 * i1);
        }
        fetch_s += kGroups;
        if (fetch_s >= stop) fetch_s = begin, ++fetch_n;
    };
    // ---- the token at work, and its sines and cosines
    int pos = -1;
    int64_t cache_off = -1, exp_off = 0, t = t0;
    float2 cs[4], sn[4], ns[4];  // of pairs 2 i, 2 i + 1; ns = -sn
    auto begin_token = [&](int n) {
        if (n % 32 == 0) look(n);
        pos = __shfl_sync(0xffffffffu, found.pos, n % 32);
        cache_off = __shfl_sync(0xffffffffu, found.cache_off, n % 32);
        if constexpr (kForm != kRows16) exp_off = __shfl_sync(0xffffffffu, found.exp_off, n % 32);
        t = t0 + n * step;
        if (pos < 0 || !p.rot) return;
        // the groups of lanes need the same 8 a lane: each makes some of them
        constexpr int kOwn = kGroups < 8 ? 8 / kGroups : 1;
        const int64_t at = p.positions ? p.positions[t] : pos;
        float s[kOwn], c8[kOwn];
#pragma unroll
        for (int e = 0; e < kOwn; ++e) {
            const int k = (gr * kOwn + e) % 8, i = min(kInterleaved ? (k < 4 ? i0 / 2 + k : i1 / 2 + k - 4) : 8 * li + k, p.rot / 2 - 1);
            turn_sincos((uint32_t)(((uint64_t)at * turns[i]) >> 32), &s[e], &c8[e]);
            s[e] *= p.magnitude;
            c8[e] *= p.magnitude;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            (i % 2 ? sn[i / 2].y : sn[i / 2].x) = __shfl_sync(0xffffffffu, s[i % kOwn], i / kOwn * kLanes + li);
            (i % 2 ? cs[i / 2].y : cs[i / 2].x) = __shfl_sync(0xffffffffu, c8[i % kOwn], i / kOwn * kLanes + li);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) ns[i] = make_float2(-sn[i].x, -sn[i].y);
    };
    // a lane's 16 elements as pairs: `one` the first and `two` the second elements of pairs 2 i, 2 i + 1. Half layout: the
    // elements of the first pack, of the second; interleaved: the even ones, the odd ones.
    auto unpack = [&](const uint4 (&in)[2], float2 (&one)[4], float2 (&two)[4]) {
        const uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = widen2<kBf16>(kInterleaved ? w[2 * i] : w[i]), g = widen2<kBf16>(kInterleaved ? w[2 * i + 1] : w[4 + i]);
            one[i] = kInterleaved ? make_float2(f.x, g.x) : f;
            two[i] = kInterleaved ? make_float2(f.y, g.y) : g;
        }
    };
    auto turn = [&](float2 (&one)[4], float2 (&two)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (kInterleaved && !(i < 2 ? turned0 : turned1)) continue;
            const float2 a = one[i], b = two[i];
            one[i] = fma2(a, cs[i], mul2(b, ns[i]));
            two[i] = fma2(b, cs[i], mul2(a, sn[i]));
        }
    };
    // the first (k = 0) or second pack's elements in order
    auto pack = [&](const float2 (&one)[4], const float2 (&two)[4], int k, float2 (&x)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 2 * k + i / 2;
            if constexpr (kInterleaved) x[i] = i % 2 ? make_float2(one[j].y, two[j].y) : make_float2(one[j].x, two[j].x);
            else x[i] = k ? two[i] : one[i];
        }
    };
    auto turn_words = [&](uint4 (&in)[2]) {
        float2 one[4], two[4], x[4];
        unpack(in, one, two);
        turn(one, two);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            pack(one, two, k, x);
            in[k] = make_uint4(pack2<kBf16>(x[0].x, x[0].y), pack2<kBf16>(x[1].x, x[1].y), pack2<kBf16>(x[2].x, x[2].y), pack2<kBf16>(x[3].x, x[3].y));
        }
    };
    // ---- a round of the token's rows s + gr
    auto work = [&](uint4 (&in)[2], int s) {
        if (s < q_slots) {
            const int r = s + gr;
            if (pos < 0 || r >= p.heads || r >= stop) return;
            char* dst = p.q_out + t * p.qos[0] + r * p.qos[1];
            if (turned0) turn_words(in);
            if (on0) *reinterpret_cast<uint4*>(dst + 2 * i0) = in[0];
            if (on1) *reinterpret_cast<uint4*>(dst + 2 * i1) = in[1];
            return;
        }
        if (pos < 0 || cache_off < 0) return;  // (of the whole warp)
        const int r = s - q_slots + gr, h = r >= c.hkv ? r - c.hkv : r;
        const bool there = s + gr < stop, v = r >= c.hkv, turns = turned0 && !v;  // (no lane turns its second pack alone)
        char* dst = (v ? c.v : c.k) + cache_off + h * c.head_stride;
        if constexpr (kForm == kRows16) {
            if (!there) return;
            if (turns) turn_words(in);
            if (on0) *reinterpret_cast<uint4*>(dst + 2 * i0) = in[0];
            if (on1) *reinterpret_cast<uint4*>(dst + 2 * i1) = in[1];
        } else {
            const uint32_t p0 = pack_max(in[0]), p1 = pack_max(in[1]);
            const int e = row_exp<kForm>(row_max<kBf16, kLanes>(in, __vmaxu2(p0, p1)), !v && p.rot ? p.grow + (kForm == kRowsE4m3) : 0);
            const float inv = exp2_of(-e);
            float2 one[4], two[4], x[2][4];
            unpack(in, one, two);
            if (turns) turn(one, two);
            if constexpr (kForm == kRowsE4m3) {
#pragma unroll
                for (int j = 0; j < 4; ++j) one[j] = mul2(one[j], make_float2(inv, inv)), two[j] = mul2(two[j], make_float2(inv, inv));
            }
            pack(one, two, 0, x[0]);
            pack(one, two, 1, x[1]);
            const int64_t byte = exp_off + (int64_t)h * c.page_size;
            if (there && li == 0) (v ? c.v_exp : c.k_exp)[byte] = (uint8_t)(e + 127);
            if constexpr (kForm == kRowsE4m3) {
                if (!there) return;
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (k ? on1 : on0)
                        *reinterpret_cast<uint2*>(dst + (k ? i1 : i0)) =
                            make_uint2(to_e4m3x2(x[k][0].x, x[k][0].y) | to_e4m3x2(x[k][1].x, x[k][1].y) << 16,
                                       to_e4m3x2(x[k][2].x, x[k][2].y) | to_e4m3x2(x[k][3].x, x[k][3].y) << 16);
            } else {
                uint32_t m0, m1;
                if (turns) {
                    m0 = max_bits(x[0]);
                    m1 = max_bits(x[1]);
                } else {
                    m0 = __float_as_uint(magnitude_of<kBf16>(max(p0 & 0xffffu, p0 >> 16)));
                    m1 = __float_as_uint(magnitude_of<kBf16>(max(p1 & 0xffffu, p1 >> 16)));
                }
                if (apart) {  // of the whole call
                    const uint32_t a0 = __shfl_sync(0xffffffffu, m0, from0), b0 = __shfl_sync(0xffffffffu, m1, from0);
                    const uint32_t a1 = __shfl_sync(0xffffffffu, m0, from1), b1 = __shfl_sync(0xffffffffu, m1, from1);
                    m0 = max(m0, second0 ? b0 : a0);
                    m1 = max(m1, second1 ? b1 : a1);
                } else {
                    m0 = m1 = max(m0, m1);
                }
                if (!there) return;
                const uint32_t s0 = group_scale(m0, inv), s1 = apart ? group_scale(m1, inv) : s0;
                uint8_t* scales = (v ? c.v_scale : c.k_scale) + byte * (c.d / 16);
                const float power = exp2_of(e);
                const uint2 codes = make_uint2(group_codes(x[0], s0, power, inv, reciprocal), group_codes(x[1], s1, power, inv, reciprocal));
                if (!apart) {
                    if (on0) {
                        *reinterpret_cast<uint2*>(dst + i0 / 2) = codes;
                        scales[i0 / 16] = (uint8_t)s0;
                    }
                } else {
                    if (on0) {
                        *reinterpret_cast<uint32_t*>(dst + i0 / 2) = codes.x;
                        if (i0 % 16 == 0) scales[i0 / 16] = (uint8_t)s0;
                    }
                    if (on1) {
                        *reinterpret_cast<uint32_t*>(dst + i1 / 2) = codes.y;
                        if (i1 % 16 == 0) scales[i1 / 16] = (uint8_t)s1;
                    }
                }
            }
        }
    };
    uint4 in[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(in[u]);
    for (int n = 0, s = begin;;) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (s == begin) {
                if (n == tokens) return;
                begin_token(n);
            }
            uint4 now[2] = {in[u][0], in[u][1]};
            if (kAhead > 1) fetch(in[u]);
            work(now, s);
            if (kAhead == 1) fetch(in[u]);
            s += kGroups;
            if (s >= stop) s = begin, ++n;
        }
    }
}

template <bool kBf16, int kForm, bool kInterleaved, int kLanes>
cudaError_t launch_lanes(const RopeAppendParams& p, cudaStream_t stream) {
    // Rounds ahead, GB300: prompts of 91 K tokens in e4m3 2 170 us, 3 164; 4-bit ones 94 and 102; 16-bit ones 57 and 61.
    constexpr int kGroups = 32 / kLanes, kAhead = kForm == kRowsE4m3 ? 3 : 2;
    const int slots = (p.heads + kGroups - 1) / kGroups * kGroups + 2 * p.rows.c.hkv;
    const int64_t blocks = (p.rows.tokens + kWarps - 1) / kWarps;
    // Whole tokens, as many warps as are resident; with few tokens one round of a token's rows a warp.
    if (blocks >= 152 * 2)
        return launch_early(rope_append_kernel<kBf16, kForm, kInterleaved, kLanes, kAhead>, dim3((unsigned)std::min<int64_t>(blocks, 152 * kPerSm)),
                            dim3(kWarps * 32), 0, stream, p, slots);
    return launch_early(rope_append_kernel<kBf16, kForm, kInterleaved, kLanes, 1>, dim3((unsigned)blocks, (unsigned)((slots + kGroups - 1) / kGroups)),
                        dim3(kWarps * 32), 0, stream, p, kGroups);
}

template <bool kBf16, int kForm, bool kInterleaved>
cudaError_t launch_layout(const RopeAppendParams& p, cudaStream_t stream) {
    if (p.rows.c.d <= 32) return launch_lanes<kBf16, kForm, kInterleaved, 2>(p, stream);
    if (p.rows.c.d <= 64) return launch_lanes<kBf16, kForm, kInterleaved, 4>(p, stream);
    return launch_lanes<kBf16, kForm, kInterleaved, 8>(p, stream);
}

template <int kForm>
cudaError_t launch_form(const RopeAppendParams& p, cudaStream_t stream) {
    if (p.rows.c.dtype == kBf16)
        return p.interleaved ? launch_layout<true, kForm, true>(p, stream) : launch_layout<true, kForm, false>(p, stream);
    return p.interleaved ? launch_layout<false, kForm, true>(p, stream) : launch_layout<false, kForm, false>(p, stream);
}

}  // namespace
}  // namespace fa2
