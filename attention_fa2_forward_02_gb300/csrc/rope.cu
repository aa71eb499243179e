// rope.cu - rotary positions on [b, h, n, d] views, forward and backward.
//
// y1 = m (x1 cos a - x2 sin a), y2 = m (x2 cos a + x1 sin a) with a = position * inv_freq[i] for
// pair i of the rotated elements; the backward is the same with -a.
//
// The angle: only its fraction of a turn matters, and at position 2^20 a float32 product has
// already lost a sixteenth of a radian. f / (2 pi) is turned into a 64-bit fixed-point fraction
// (integers only: this part's float64 rate is a hundredth of its integer rate) and multiplied by the position
// modulo 2^64, which keeps the fraction exact to position * 2^-64; the fixed-point frequencies are
// made once per block, in shared memory. The upper 32 bits of a product, as a signed fraction of
// a turn, lose their nearest quarter turn as an integer, exactly, and what is left, at most an
// eighth, goes into the Taylor sums of sine and cosine in float32 (turn_sincos). GB300, bf16,
// d = 128: B=2 H=16 N=2048 7.7 us, and 8.0 with sincospif; B=64 H=1 N=4096, where every sine is used
// once, 35.7 and 39.2; the special function unit's sine and cosine, within 2^-20.9 only, 7.4 and 30.5.
//
// Each thread owns P pairs of one token (two 16-byte vectors where sizes and strides allow) and
// walks over heads, two of them in flight: the P sines and cosines are made once for all of them,
// while the first heads are being read. Bound by memory: 134 MB (B=2 H=16 N=8192 d=128, bf16) in
// 22.3 us, 6.0 TB/s.
#include "common.cuh"
#include "internal.h"

namespace fa2 {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 2;    // heads in flight per thread
constexpr int kMaxHeads = 4;  // heads a thread walks over

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

template <int kBytes>
struct Word;
template <>
struct Word<16> { using T = uint4; };
template <>
struct Word<8> { using T = uint2; };
template <>
struct Word<4> { using T = uint32_t; };
template <>
struct Word<2> { using T = uint16_t; };

template <typename E>
__device__ __forceinline__ float widen(E x);
template <>
__device__ __forceinline__ float widen(float x) { return x; }
template <>
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename E>
__device__ __forceinline__ E narrow(float x);
template <>
__device__ __forceinline__ float narrow(float x) { return x; }
template <>
__device__ __forceinline__ __half narrow(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow(float x) { return __float2bfloat16_rn(x); }

template <typename E, int P>
union Pack {
    typename Word<P * sizeof(E)>::T w;
    E e[P];
    __device__ Pack() {}
};

// None of the inputs is declared __restrict__: the kernel before may still be writing them while this
// one is set up, and such loads need not stay behind the wait.
//
// A thread's two packs of P elements: for the half layout the packs at i and i + rot / 2, for
// the interleaved one the 2 P elements from 2 i.
template <typename E, int P, bool kInterleaved>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const E* x, E* y, const int32_t* positions, int64_t position_stride,
                const double* inv_freq, int n_tokens, int heads, int heads_per_thread, int chunks, int d, int rot,
                int64_t xb, int64_t xh, int64_t xn, int64_t yb, int64_t yh, int64_t yn, float magnitude, int backward) {
    using W = typename Word<P * sizeof(E)>::T;
    const int b = blockIdx.y / chunks, chunk = blockIdx.y % chunks;
    __shared__ uint64_t turns[512];
    const int n = blockIdx.x * blockDim.y + threadIdx.y;
    grid_begin();
    for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < rot / 2; i += blockDim.x * blockDim.y) turns[i] = turns_of(inv_freq[i]);
    __syncthreads();
    if (n >= n_tokens) return;
    const int h0 = chunk * heads_per_thread, h1 = min(heads, h0 + heads_per_thread);
    const bool in_place = x == y;
    const int rot_units = rot / (2 * P), units = rot_units + (in_place ? 0 : (d - rot + 2 * P - 1) / (2 * P));
    const E* xr = x + b * xb + n * xn;
    E* yr = y + b * yb + n * yn;
    for (int u = threadIdx.x; u < units; u += blockDim.x) {
        const bool rotates = u < rot_units;  // else elements that do not rotate: one or two packs, copied
        const int i0 = rotates ? (kInterleaved ? 2 * P * u : P * u) : rot + (u - rot_units) * 2 * P;
        const int i1 = rotates && !kInterleaved ? i0 + rot / 2 : i0 + P;
        const bool both = i1 < d;
        Pack<E, P> a[kUnroll], g[kUnroll];
        auto fetch = [&](int h) {
#pragma unroll
            for (int k = 0; k < kUnroll; ++k)
                if (h + k < h1) {
                    a[k].w = *reinterpret_cast<const W*>(xr + (h + k) * xh + i0);
                    if (both) g[k].w = *reinterpret_cast<const W*>(xr + (h + k) * xh + i1);
                }
        };
        fetch(h0);  // on their way while the angles are made
        float c[P], s[P];
        if (rotates) {
            const int64_t pos = positions ? positions[b * position_stride + n] : n;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                turn_sincos((uint32_t)(((uint64_t)pos * turns[P * u + p]) >> 32), &s[p], &c[p]);
                c[p] *= magnitude;
                s[p] *= backward ? -magnitude : magnitude;
            }
        }
        for (int h = h0;;) {
#pragma unroll
            for (int k = 0; k < kUnroll; ++k)
                if (h + k < h1) {
                    Pack<E, P> o0, o1;
                    o0.w = a[k].w;
                    o1.w = g[k].w;
                    if (rotates) {
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            // pair p: elements p of the two packs, or elements 2 p, 2 p + 1 of both in a row
                            const int q = kInterleaved ? 2 * p : p;
                            const float x1 = widen<E>(q < P ? a[k].e[q % P] : g[k].e[q % P]);
                            const float x2 = widen<E>(kInterleaved ? (q + 1 < P ? a[k].e[(q + 1) % P] : g[k].e[(q + 1) % P])
                                                                   : g[k].e[p]);
                            const E y1 = narrow<E>(x1 * c[p] - x2 * s[p]), y2 = narrow<E>(x2 * c[p] + x1 * s[p]);
                            if (kInterleaved) {
                                (q < P ? o0.e[q % P] : o1.e[q % P]) = y1;
                                (q + 1 < P ? o0.e[(q + 1) % P] : o1.e[(q + 1) % P]) = y2;
                            } else {
                                o0.e[p] = y1;
                                o1.e[p] = y2;
                            }
                        }
                    }
                    *reinterpret_cast<W*>(yr + (h + k) * yh + i0) = o0.w;
                    if (both) *reinterpret_cast<W*>(yr + (h + k) * yh + i1) = o1.w;
                }
            h += kUnroll;
            if (h >= h1) break;
            fetch(h);
        }
    }
}

template <typename E, int P>
cudaError_t launch_p(const RopeParams& p, cudaStream_t stream) {
    const int units = p.rot / (2 * P) + (p.x == p.y ? 0 : (p.d - p.rot + 2 * P - 1) / (2 * P));
    const int ux = units < kThreads ? units : kThreads;
    const int ty = kThreads / ux;
    const int64_t blocks_x = (p.n + ty - 1) / ty;
    // Heads per thread: up to kMaxHeads, in equal parts, while that leaves every SM threads enough to
    // hide the loads, else fewer (each part of the heads makes the angles again). GB300, B=2 H=16
    // N=8192 d=128: 4 heads a thread 22.2 us, 8 22.6, 2 23.5; B=3 H=20 N=5003 d=96 with 32 turning:
    // 4 20.6 us, 8 21.1, 2 22.4.
    int64_t chunks = (p.h + kMaxHeads - 1) / kMaxHeads;
    while (chunks < p.h && blocks_x * p.b * chunks < (int64_t)152 * 8) chunks *= 2;
    int hpt = (int)((p.h + chunks - 1) / chunks);
    if (hpt > kUnroll) hpt = (hpt + kUnroll - 1) / kUnroll * kUnroll;  // whole rounds
    chunks = (p.h + hpt - 1) / hpt;
    auto kern = p.interleaved ? rope_kernel<E, P, true> : rope_kernel<E, P, false>;
    for (int64_t b0 = 0; b0 < p.b;) {  // grid.y holds at most 65535 (batch entry, part of the heads)
        int64_t nb = 65535 / chunks;
        if (nb < 1) {
            hpt = (int)((p.h + 65534) / 65535);
            chunks = (p.h + hpt - 1) / hpt;
            nb = 1;
        }
        if (nb > p.b - b0) nb = p.b - b0;
        const cudaError_t e = launch_early(
            kern, dim3((unsigned)blocks_x, (unsigned)(nb * chunks)), dim3(ux, ty), 0, stream, static_cast<const E*>(p.x) + b0 * p.xs[0],
            static_cast<E*>(p.y) + b0 * p.ys[0], p.positions ? p.positions + b0 * p.position_stride : nullptr, p.position_stride,
            p.inv_freq, (int)p.n, (int)p.h, hpt, (int)chunks, p.d, p.rot, p.xs[0], p.xs[1], p.xs[2], p.ys[0], p.ys[1], p.ys[2],
            p.magnitude, (int)p.backward);
        if (e != cudaSuccess) return e;
        b0 += nb;
    }
    return cudaSuccess;
}

// The widest pack that the rotated half, the head and every stride are whole multiples of.
template <typename E>
cudaError_t launch_e(const RopeParams& p, cudaStream_t stream) {
    auto fits = [&](int P) {
        bool ok = (p.rot / 2) % P == 0 && p.d % P == 0;
        for (int i = 0; i < 3; ++i) ok = ok && p.xs[i] % P == 0 && p.ys[i] % P == 0;
        return ok;
    };
    if constexpr (sizeof(E) == 2)
        if (fits(8)) return launch_p<E, 8>(p, stream);
    if (fits(4)) return launch_p<E, 4>(p, stream);
    if (fits(2)) return launch_p<E, 2>(p, stream);
    return launch_p<E, 1>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
    switch (p.dtype) {
        case kF32: return launch_e<float>(p, stream);
        case kF16: return launch_e<__half>(p, stream);
        default: return launch_e<__nv_bfloat16>(p, stream);
    }
}

}  // namespace fa2
