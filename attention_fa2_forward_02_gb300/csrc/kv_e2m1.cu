// kv_e2m1.cu - 4-bit rows out of the pages of a cache, and which kernels write new ones (kv_rope.cuh).
#include "paged.cuh"

namespace fa2 {
namespace {

constexpr int kWarps = 4;

// 4-bit rows back to 16 bits: as kv_rows_kernel of kv_cache.cu, a lane's 16 elements as packs of 8 that lie kLanes
// packs apart, so that both sides of a row's lanes are one after another in memory. Every element is exact in bfloat16. GB300,
// 9 sequences of up to 16384, 8 heads of 128 (425 MB, 7 bytes written for 2 read): 70 us, 6.1 TB/s; a step's 2.9 us.
template <bool kBf16, int kLanes, int kRows, int kTok>
__global__ void __launch_bounds__(kWarps * 32) kv_read_e2m1_kernel(const KvRowsParams p, int rows_per_warp) {
    const PagedParams& c = p.c;
    constexpr int kGroups = 32 / kLanes;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * kTok;
    const int b = blockIdx.z;
    grid_begin();
    const int len = bounded_len(c.lens[b], c.room, c.status);
    if (t0 >= p.tokens || t0 >= len) return;
    int64_t my_off = -1, my_exp = -1;
    {
        const int64_t pos = t0 + lane % kTok;
        if (pos < p.tokens && pos < len) {
            const int at = page_of(c, (int)pos);
            const Slot s = slot_of(c, c.table[b * c.table_stride + at], (int)pos - at * c.page_size);
            my_off = s.off;
            my_exp = s.exp;
        }
    }
    const int li = lane % kLanes, gr = lane / kLanes;
    const int total = 2 * c.hkv, begin = blockIdx.y * rows_per_warp, stop = min(total, begin + rows_per_warp);
    for (int n = 0; n < kTok; ++n) {
        const int64_t cache_off = __shfl_sync(0xffffffffu, my_off, n), exp_off = __shfl_sync(0xffffffffu, my_exp, n);
        if (cache_off < 0) continue;
        for (int r0 = begin + gr; r0 - gr < stop; r0 += kGroups * kRows) {
            uint32_t codes[kRows][2], scale[kRows][2], byte[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int r = r0 + i * kGroups, h = r >= c.hkv ? r - c.hkv : r;
                if (r >= stop) continue;
                const bool v = r >= c.hkv;
                const char* src = (v ? c.v : c.k) + cache_off + h * c.head_stride;
                const int64_t e = exp_off + (int64_t)h * c.page_size;
                const uint8_t* scales = (v ? c.v_scale : c.k_scale) + e * (c.d / 16);
                byte[i] = (v ? c.v_exp : c.k_exp)[e];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int pack = li + k * kLanes;
                    if (8 * pack >= c.d) continue;
                    codes[i][k] = *reinterpret_cast<const uint32_t*>(src + 4 * pack);
                    scale[i][k] = scales[pack / 2];
                }
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int r = r0 + i * kGroups, h = r >= c.hkv ? r - c.hkv : r;
                if (r >= stop) continue;
                const bool v = r >= c.hkv;
                char* dst = v ? p.v + b * p.vs[0] + h * p.vs[1] + (t0 + n) * p.vs[2] : p.k + b * p.ks[0] + h * p.ks[1] + (t0 + n) * p.ks[2];
                const float two = __uint_as_float(byte[i] << 23);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int pack = li + k * kLanes;
                    if (8 * pack >= c.d) continue;
                    uint32_t f[4], o[4];
                    e2m1x8_to_f16x8(codes[i][k], f);
                    const uint32_t s = e4m3x2_to_f16x2(scale[i][k] * 0x101u);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t x = hmul2(f[j], s);  // exact: 6 bits
                        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x));
                        o[j] = pack2<kBf16>(y.x * two, y.y * two);
                    }
                    *reinterpret_cast<uint4*>(dst + 16 * pack) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }
}

template <bool kBf16, int kLanes>
cudaError_t launch_read(const KvRowsParams& p, cudaStream_t stream) {
    constexpr int kGroups = 32 / kLanes, kRows = 4, kTok = 2;
    const int total = 2 * p.c.hkv;
    const unsigned batch = (unsigned)p.c.batch;
    auto blocks = [&](int tok) { return (p.tokens + kWarps * tok - 1) / (kWarps * tok); };
    if (blocks(kTok) * batch >= 152 * 8) {
        const dim3 grid((unsigned)blocks(kTok), 1, batch);
        return launch_early(kv_read_e2m1_kernel<kBf16, kLanes, kRows, kTok>, grid, dim3(kWarps * 32), 0, stream, p, total);
    }
    const dim3 grid((unsigned)blocks(1), (unsigned)((total + kGroups - 1) / kGroups), batch);
    return launch_early(kv_read_e2m1_kernel<kBf16, kLanes, 1, 1>, grid, dim3(kWarps * 32), 0, stream, p, kGroups);
}

template <bool kBf16>
cudaError_t launch_read_lanes(const KvRowsParams& p, cudaStream_t stream) {
    if (p.c.d <= 32) return launch_read<kBf16, 2>(p, stream);
    if (p.c.d <= 64) return launch_read<kBf16, 4>(p, stream);
    return launch_read<kBf16, 8>(p, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams& p, cudaStream_t stream) {
    switch (p.rows.c.form) {
        case kRows16: return launch_rope_append_16(p, stream);
        case kRowsE4m3: return launch_rope_append_e4m3(p, stream);
        default: return launch_rope_append_e2m1(p, stream);
    }
}

cudaError_t launch_kv_read_e2m1(const KvRowsParams& p, cudaStream_t stream) {
    return p.c.dtype == kBf16 ? launch_read_lanes<true>(p, stream) : launch_read_lanes<false>(p, stream);
}

}  // namespace fa2
