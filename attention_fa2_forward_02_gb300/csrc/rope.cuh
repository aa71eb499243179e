// rope.cuh - angles of rotary positions: fractions of a turn in fixed point, and their sines and cosines.
#pragma once

#include <stdint.h>

namespace fa2 {

// f / (2 pi) modulo 1 in units of 2^-64, for finite f.
__device__ __forceinline__ uint64_t turns_of(double f) {
    const uint64_t bits = (uint64_t)__double_as_longlong(f);
    const int e = (int)((bits >> 52) & 0x7ff) - 1023;  // |f| = M 2^(e - 63), M's top bit set
    const uint64_t m = (bits << 11) | (1ull << 63);
    constexpr uint64_t kInv2Pi66 = 0xA2F9836E4E44152Aull;  // 2^66 / (2 pi)
    const uint64_t hi = __umul64hi(m, kInv2Pi66);          // |f| / (2 pi) = hi 2^(e - 65)
    uint64_t t;
    if (e <= 1) t = 1 - e < 64 ? hi >> (1 - e) : 0;  // (zero and subnormal f land here: 0)
    else t = e - 1 < 64 ? hi << (e - 1) : 0;
    return (bits >> 63) ? 0 - t : t;
}

// sin and cos of t 2^-32 turns. a = 2 pi 2^-32 (t - q 2^30) lies within pi / 4; the sums' next terms
// are a^11 / 11! < 2^-29 and a^10 / 10! < 2^-25. With u = 2^-24 a's own error is 3 u |a|, the sine's
// 2.8 u in all, the cosine's 3.4 u.
__device__ __forceinline__ void turn_sincos(uint32_t t, float* s, float* c) {
    const uint32_t q = (t + (1u << 29)) >> 30;
    const float a = (float)(int32_t)(t - (q << 30)) * (6.28318530717958648f * 0x1p-32f), z = a * a;
    const float sn = fmaf(a * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), a);
    const float cs = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 40320, -1.f / 720), 1.f / 24), -0.5f), 1.f);
    const float s1 = q & 1 ? cs : sn, c1 = q & 1 ? sn : cs;
    *s = __uint_as_float(__float_as_uint(s1) ^ (q & 2) << 30);
    *c = __uint_as_float(__float_as_uint(c1) ^ ((q + 1) & 2) << 30);
}

}  // namespace fa2
