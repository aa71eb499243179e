// fa2_decode.cu - attention of one new token of each sequence over a paged key-value cache.
//
// fa2_forward's formula for one query row a head: O = softmax(scale q K^T) V, LSE, over the
// sequence's cached keys. Every key and value is read once for up to 16 query heads, 4 * 16
// FLOPs for 4 bytes at most, so memory sets the pace and the products only have to keep up:
// they run as warp-level 16 x 8 x 16 products on registers, whose 16 rows are the query heads
// of one key-value head. (The 128-row products of the tensor memory path would want 128 rows
// of queries, or the keys as rows and then the probabilities through shared memory.)
//
// Work: the keys of every (sequence, key-value head, 16 query heads) item are cut into blocks
// of kKeys; all blocks of all items in a row are divided evenly over the CTAs, whatever the
// lengths, and a CTA's blocks of one item over its warps, one by one. Each warp keeps its own
// running maximum, sum and O, and its own ring of stages filled by asynchronous 16-byte copies:
// no barrier joins the warps until the item ends. There the CTA adds its warps' results up in
// shared memory; an item that lies in one CTA is then done, the others leave (m, l, O) in the
// workspace, at most two per CTA, and the second kernel joins them in CTA order.
//
// The 8-bit cache: with key scale 2^a and value scale 2^e per row, the score of a key is
// x = scale log2(e) 2^a (q . codes) + e, its weight P = 2^(x - m) with m a maximum of x: the
// value's scale is inside the weight, the second product runs on bare codes, and
// l = sum P 2^-e counts the softmax's own terms. Codes are exact in half; q (bfloat16) is
// brought to half exactly by a power of two of its row's largest element.
#include "paged.cuh"

namespace fa2 {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;        // query heads per item
constexpr int kMaxCtas = 152;    // CTAs of the first kernel (a fixed number: the split depends on the lengths alone)
constexpr float kRescale = 8.0f; // the running maximum may lag by this much (base-2 units) before O is rescaled
constexpr float kLn2 = 0.693147180559945309f;

template <int D, bool kE4m3>
struct Cfg {
    static constexpr int kKeys = 16;                        // keys per block
    static constexpr int kRowBytes = kE4m3 ? D : 2 * D;
    static constexpr int kChunks = kRowBytes / 16;          // 16-byte chunks a row
    static constexpr int kTile = kKeys * kRowBytes;         // K or V of a block
    static constexpr int kInfo = kKeys * 16;                // float4 per key
    static constexpr int kStage = 2 * kTile + kInfo;
    static constexpr int kMerge = kRows * (D + 4) * 4;      // a warp's O, m, l at the end of an item
    static constexpr int kStagesWanted = kMerge / kStage + 1 > 4 ? kMerge / kStage + 1 : 4;
    static constexpr int kStages = kWarps * kStage * kStagesWanted <= 220 * 1024 ? kStagesWanted : 3;
    static constexpr int kWarpBytes = kStages * kStage > kMerge ? kStages * kStage : kMerge;
    static constexpr int kSmem = kWarps * kWarpBytes + 64;
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

// Position of chunk `c` of row `r` in a tile: the eight rows an ldmatrix reads at one chunk lie
// in eight different 16-byte bank groups.
template <int kChunks>
__device__ __forceinline__ int swizzle(int r, int c) {
    if constexpr (kChunks >= 8) return r * kChunks + (c ^ (r & 7));
    else if constexpr (kChunks == 4) return r * 4 + (c ^ ((r >> 1) & 3));
    else return r * 2 + (c ^ ((r >> 2) & 1));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
    const int bytes = on ? 16 : 0;  // 0: the 16 bytes are filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kBf16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// How the blocks of all items are divided over the CTAs. Items are ordered by (sequence, head
// block); every sequence has `per_seq` of them, with the same number of blocks.
struct Split {
    int64_t total;  // blocks in all
    int64_t ctas;   // CTAs that have any: at least a block for each of their warps
    __device__ __forceinline__ int64_t begin(int64_t c) const { return c * total / ctas; }
    // the CTA that block u belongs to: the largest c with begin(c) <= u
    __device__ __forceinline__ int64_t owner(int64_t u) const {
        int64_t c = u * ctas / total;
        while (c + 1 < ctas && begin(c + 1) <= u) ++c;
        while (c > 0 && begin(c) > u) --c;
        return c;
    }
};

__device__ __forceinline__ Split split_of(int64_t total, int max_ctas) {
    Split s;
    s.total = total;
    s.ctas = (total + kWarps - 1) / kWarps;
    if (s.ctas > max_ctas) s.ctas = max_ctas;
    return s;
}

// The keys [first, len) of sequence b that the window leaves.
struct Range {
    int first, len;
};
__device__ __forceinline__ Range range_of(const DecodeParams& p, int b) {
    const int len = bounded_len(p.c.lens[b], p.c.room, p.c.status);
    const int first = p.window > 0 && len > p.window ? (int)(len - p.window) : 0;
    return {first, len};
}
template <int kKeys>
__device__ __forceinline__ int blocks_of(Range r) { return (r.len - r.first + kKeys - 1) / kKeys; }

// Sum over the CTA's threads, the same value for each (scratch: 8 int64, free again on return).
__device__ __forceinline__ int64_t cta_sum(int64_t v, int64_t* scratch, int warps) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    int64_t t = 0;
    for (int i = 0; i < warps; ++i) t += scratch[i];
    __syncthreads();
    return t;
}

// Workspace: per CTA two partial results (its first item, if that began before it or ends after
// it; its last item, if that ends after it), each [kRows][D] floats and then [kRows] (m, l).
template <int D>
__device__ __forceinline__ float* partial(float* ws, int64_t cta, int which) {
    return ws + (cta * 2 + which) * (kRows * (D + 2));
}

template <int D, bool kBf16, bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1) fa2_decode_kernel(const DecodeParams p) {
    using C = Cfg<D, kE4m3>;
    constexpr bool kMmaBf16 = kBf16 && !kE4m3;
    constexpr int kKeys = C::kKeys, S = C::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    int64_t* scratch = reinterpret_cast<int64_t*>(smem + kWarps * C::kWarpBytes);
    const PagedParams& c = p.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = p.heads / c.hkv, hblocks = (group + kRows - 1) / kRows;
    const int64_t per_seq = (int64_t)c.hkv * hblocks;

    int64_t mine = 0;
    for (int b = threadIdx.x; b < c.batch; b += kThreads) mine += blocks_of<kKeys>(range_of(p, b));
    const Split split = split_of(cta_sum(mine, scratch, kWarps) * per_seq, gridDim.x);
    if ((int64_t)blockIdx.x >= split.ctas) return;
    const int64_t u_begin = split.begin(blockIdx.x), u_end = split.begin(blockIdx.x + 1);

    // the sequence that block u_begin lies in
    int b = 0;
    int64_t u_seq = 0;  // first block of sequence b
    {
        int64_t before = 0;
        int b0 = 0;
        for (;; b0 += kThreads) {  // whole strips of kThreads sequences, then the one inside
            const int bi = b0 + threadIdx.x;
            const int64_t v = bi < c.batch ? blocks_of<kKeys>(range_of(p, bi)) * per_seq : 0;
            const int64_t strip = cta_sum(v, scratch, kWarps);
            if (before + strip > u_begin) break;
            before += strip;
        }
        b = b0;
        u_seq = before;
        for (;;) {
            const int64_t v = blocks_of<kKeys>(range_of(p, b)) * per_seq;
            if (u_seq + v > u_begin) break;
            u_seq += v;
            ++b;
        }
    }

    uint8_t* my = smem + warp * C::kWarpBytes;
    const uint32_t my_addr = smem_u32(my);
    const int g = lane >> 2, t = lane & 3;  // row (head) and column group in the products' fragments
    bool first_item = true;

    for (int64_t u = u_begin; u < u_end;) {
        // ---- the item that block u lies in, and this CTA's blocks [k0, k1) of it
        Range range = range_of(p, b);
        int nb = blocks_of<kKeys>(range);
        while (u >= u_seq + nb * per_seq) {
            u_seq += nb * per_seq;
            range = range_of(p, ++b);
            nb = blocks_of<kKeys>(range);
        }
        const int64_t item = (u - u_seq) / nb;
        const int64_t u_item = u_seq + item * nb;
        const int hk = (int)(item / hblocks), hb = (int)(item % hblocks);
        const int k0 = (int)(u - u_item);
        const int k1 = (int)(u_end - u_item < nb ? u_end - u_item : nb);
        const int head0 = hk * group + hb * kRows;               // first query head
        const int rows = min(kRows, group - hb * kRows);         // query heads of the item

        // ---- q as the first product's left operand: rows g and g + 8
        uint32_t qf[D / 16][4];
        float qscale[2] = {1.f, 1.f};
        {
            const uint16_t* qb = static_cast<const uint16_t*>(p.q) + b * p.q_batch;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = g + 8 * half;
                const uint16_t* qr = qb + (int64_t)(head0 + r) * p.q_head;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    // elements 2t, 2t+1 and 2t+8, 2t+9 of 16 (8-bit cache: 4t .. 4t+3, the order its codes come in)
                    const int d0 = 16 * kk + (kE4m3 ? 4 * t : 2 * t), d1 = d0 + (kE4m3 ? 2 : 8);
                    qf[kk][half] = r < rows && d0 < c.d ? *reinterpret_cast<const uint32_t*>(qr + d0) : 0u;
                    qf[kk][2 + half] = r < rows && d1 < c.d ? *reinterpret_cast<const uint32_t*>(qr + d1) : 0u;
                }
                if constexpr (kBf16 && kE4m3) {
                    float a = 0.f;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t w = qf[kk][2 * i + half];
                            a = fmaxf(a, fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u))));
                        }
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
                    // 2^n with a 2^-n in [2^14, 2^15): half's range then reaches 2^-38 of the largest element
                    int n = (int)(__float_as_uint(a) >> 23) - 127 - 14;
                    if (a == 0.f || !(a < INFINITY)) n = 0;
                    if (n < -126) n = -126;
                    const float up = __uint_as_float((uint32_t)(127 - n) << 23);
                    qscale[half] = __uint_as_float((uint32_t)(127 + n) << 23);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t w = qf[kk][2 * i + half];
                            qf[kk][2 * i + half] =
                                pack2<false>(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
                        }
                }
                qscale[half] *= p.scale * 1.4426950408889634f;
            }
        }

        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        // ---- the ring: this warp's blocks are k0 + warp, k0 + warp + kWarps, ...
        const int n_mine = k1 - k0 > warp ? (k1 - k0 - warp + kWarps - 1) / kWarps : 0;
        const int32_t* table = c.table + b * c.table_stride;
        const int64_t head_off = hk * c.head_stride;
        // lane r < 16 looks key r of a block up; its page number is read one block ahead
        int page_next = -1;
        auto key_of = [&](int i) { return range.first + (k0 + warp + i * kWarps) * kKeys + (lane & 15); };
        auto look = [&](int i) {
            const int key = key_of(i);
            page_next = i < n_mine && key < range.len ? table[key / c.page_size] : -1;
        };
        look(0);
        auto load = [&](int i) {  // fills stage i % S with block i; always commits one group
            if (i < n_mine) {
                const int key = key_of(i);
                Slot s{-1, -1};
                if (key < range.len) s = slot_of(c, page_next, key % c.page_size);
                look(i + 1);
                const uint32_t st = my_addr + (i % S) * C::kStage;
                const int chunk = lane % C::kChunks, r0 = lane / C::kChunks;
                const bool in = chunk * 16 < c.d * (kE4m3 ? 1 : 2);
#pragma unroll
                for (int r = 0; r < kKeys; r += 32 / C::kChunks) {
                    const int64_t off = __shfl_sync(0xffffffffu, s.off, r + r0);
                    const bool on = off >= 0 && in;
                    const int64_t at = on ? off + head_off + chunk * 16 : 0;
                    const uint32_t dst = st + swizzle<C::kChunks>(r + r0, chunk) * 16;
                    cp_async16(dst, c.k + at, on);
                    cp_async16(dst + C::kTile, c.v + at, on);
                }
                if (lane < kKeys) {
                    float4 info = make_float4(1.f, s.off >= 0 ? 0.f : -INFINITY, 1.f, 0.f);
                    if constexpr (kE4m3)
                        if (s.off >= 0) {
                            const int64_t e = s.exp + (int64_t)hk * c.page_size;
                            const int ka = c.k_exp[e], ve = c.v_exp[e];
                            info.x = ka ? __uint_as_float((uint32_t)ka << 23) : 0x1p-127f;
                            info.y = (float)(ve - 127);
                            info.z = ve < 254 ? __uint_as_float((uint32_t)(254 - ve) << 23) : 0x1p-127f;
                        }
                    *reinterpret_cast<float4*>(my + (i % S) * C::kStage + 2 * C::kTile + lane * 16) = info;
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < S - 1; ++i) load(i);

        for (int i = 0; i < n_mine; ++i) {
            cp_async_wait<S - 2>();
            __syncwarp();
            load(i + S - 1);
            const uint32_t kt = my_addr + (i % S) * C::kStage, vt = kt + C::kTile;
            const float4* info = reinterpret_cast<const float4*>(my + (i % S) * C::kStage + 2 * C::kTile);
            // ---- scores of 16 keys: two 8-key column tiles
            float sc[2][4] = {};
            if constexpr (!kE4m3) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t k4[4];  // (keys 0-7, 8-15) x (d 0-7, 8-15 of this step)
                    ldsm4(kt + swizzle<C::kChunks>((lane & 7) + (lane & 16 ? 8 : 0), 2 * kk + ((lane >> 3) & 1)) * 16, k4);
                    mma16816<kMmaBf16>(sc[0], qf[kk], k4[0], k4[1]);
                    mma16816<kMmaBf16>(sc[1], qf[kk], k4[2], k4[3]);
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < D / 16; kk += 2) {
                    uint32_t k4[4];  // (keys 0-7, 8-15) x (16 codes, next 16 codes)
                    ldsm4(kt + swizzle<C::kChunks>((lane & 7) + (lane & 16 ? 8 : 0), kk + ((lane >> 3) & 1)) * 16, k4);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mma16816<false>(sc[0], qf[kk + h], e4m3x2_to_f16x2(k4[h]), e4m3x2_to_f16x2(k4[h] >> 16));
                        mma16816<false>(sc[1], qf[kk + h], e4m3x2_to_f16x2(k4[2 + h]), e4m3x2_to_f16x2(k4[2 + h] >> 16));
                    }
                }
            }
            // ---- x, the running maximum, P
            float4 inf[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) inf[j][e] = info[8 * j + 2 * t + e];
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 f = inf[j][e & 1];
                    const float s = kE4m3 ? sc[j][e] * f.x : sc[j][e];
                    sc[j][e] = fmaf(s, qscale[e >> 1], f.y);
                    mx[e >> 1] = fmaxf(mx[e >> 1], sc[j][e]);
                }
            bool grow = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                grow |= mx[h] > m[h] + kRescale || (m[h] == -INFINITY && mx[h] > -INFINITY);
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float m_new = fmaxf(m[h], mx[h]);
                    const float f = m_new == -INFINITY ? 1.f : ex2_approx(m[h] - m_new);
                    m[h] = m_new;
                    l[h] *= f;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][2 * h] *= f;
                        o[n][2 * h + 1] *= f;
                    }
                }
            }
            uint32_t pf[4];
            {
                float pr[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float mm = m[e >> 1] == -INFINITY ? 0.f : m[e >> 1];
                        pr[j][e] = ex2_approx(sc[j][e] - mm);
                        // a masked key's P is 0 whatever its factor
                        l[e >> 1] += kE4m3 ? pr[j][e] * inf[j][e & 1].z : pr[j][e];
                    }
                pf[0] = pack2<kMmaBf16>(pr[0][0], pr[0][1]);
                pf[1] = pack2<kMmaBf16>(pr[0][2], pr[0][3]);
                pf[2] = pack2<kMmaBf16>(pr[1][0], pr[1][1]);
                pf[3] = pack2<kMmaBf16>(pr[1][2], pr[1][3]);
            }
            // ---- O += P V
            if constexpr (!kE4m3) {
#pragma unroll
                for (int n = 0; n < D / 8; n += 2) {
                    uint32_t v4[4];  // (keys 0-7, 8-15) of chunk n, of chunk n + 1
                    ldsm4_t(vt + swizzle<C::kChunks>(lane & 15, n + (lane >> 4)) * 16, v4);
                    mma16816<kMmaBf16>(o[n], pf, v4[0], v4[1]);
                    mma16816<kMmaBf16>(o[n + 1], pf, v4[2], v4[3]);
                }
            } else {
#pragma unroll
                for (int n = 0; n < D / 16; n += 2) {
                    uint32_t v4[4];  // 16-code chunks n, n + 1: keys 2t, 2t+1 (and + 8) x codes 2g, 2g+1
                    ldsm4_t(vt + swizzle<C::kChunks>(lane & 15, n + (lane >> 4)) * 16, v4);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a = __byte_perm(v4[2 * h], 0, 0x3120), b8 = __byte_perm(v4[2 * h + 1], 0, 0x3120);
                        mma16816<false>(o[2 * (n + h)], pf, e4m3x2_to_f16x2(a), e4m3x2_to_f16x2(b8));
                        mma16816<false>(o[2 * (n + h) + 1], pf, e4m3x2_to_f16x2(a >> 16), e4m3x2_to_f16x2(b8 >> 16));
                    }
                }
            }
            __syncwarp();  // the stage may be filled again
        }
        cp_async_wait<0>();
        __syncwarp();

        // ---- the warps' results together, in shared memory
        float* mine_o = reinterpret_cast<float*>(my);  // [kRows][D + 4]: O, then m and l
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            const int r = g + 8 * h;
            if (r < rows) {
                float* row = mine_o + r * (D + 4);
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // columns: 8 n + 2 t + e; 8-bit cache: tiles 2 n', 2 n' + 1 hold the even and odd codes of chunk n'
                        const int d = kE4m3 ? 16 * (n >> 1) + 4 * t + 2 * e + (n & 1) : 8 * n + 2 * t + e;
                        row[d] = o[n][2 * h + e];
                    }
                if (t == 0) {
                    row[D] = m[h];
                    row[D + 1] = l[h];
                }
            }
        }
        __syncthreads();
        const bool whole = k0 == 0 && k1 == nb;
        float* part = partial<D>(p.workspace, blockIdx.x, first_item ? 0 : 1);
        for (int i = threadIdx.x; i < rows * (D / 2); i += kThreads) {
            const int r = i / (D / 2), d = i % (D / 2) * 2;
            float big = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                big = fmaxf(big, reinterpret_cast<const float*>(smem + w * C::kWarpBytes)[r * (D + 4) + D]);
            const float ref = big == -INFINITY ? 0.f : big;
            float a0 = 0.f, a1 = 0.f, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* row = reinterpret_cast<const float*>(smem + w * C::kWarpBytes) + r * (D + 4);
                const float f = ex2_approx(row[D] - ref);
                a0 += f * row[d];
                a1 += f * row[d + 1];
                sum += f * row[D + 1];
            }
            if (whole) {
                const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
                const int64_t row = (int64_t)b * p.heads + head0 + r;
                if (d < c.d)
                    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + row * c.d + d) = pack2<kBf16>(a0 * inv, a1 * inv);
                if (d == 0) p.lse[row] = sum == 0.f ? -INFINITY : (big + lg2_approx(sum)) * kLn2;
            } else {
                *reinterpret_cast<float2*>(part + r * D + d) = make_float2(a0, a1);
                if (d == 0) *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(big, sum);
            }
        }
        __syncthreads();
        first_item = false;
        u = u_item + k1;
    }
}

// Joins the items that several CTAs worked on, and writes the empty ones. One CTA per
// (sequence, item of it); thread (row, pair of columns).
template <int D, bool kBf16, int kKeys>
__global__ void __launch_bounds__(kThreads) fa2_decode_join_kernel(const DecodeParams p, int max_ctas) {
    __shared__ int64_t scratch[kWarps];
    const PagedParams& c = p.c;
    const int group = p.heads / c.hkv, hblocks = (group + kRows - 1) / kRows;
    const int64_t per_seq = (int64_t)c.hkv * hblocks;
    const int b = blockIdx.y;
    const int64_t item = blockIdx.x;
    const int hk = (int)(item / hblocks), hb = (int)(item % hblocks);
    const int head0 = hk * group + hb * kRows, rows = min(kRows, group - hb * kRows);
    int64_t all = 0, before = 0;
    for (int i = threadIdx.x; i < c.batch; i += kThreads) {
        const int64_t v = blocks_of<kKeys>(range_of(p, i));
        all += v;
        if (i < b) before += v;
    }
    const int64_t total = cta_sum(all, scratch, kWarps) * per_seq;
    before = cta_sum(before, scratch, kWarps) * per_seq;
    const int nb = blocks_of<kKeys>(range_of(p, b));
    const int64_t row0 = (int64_t)b * p.heads + head0;
    if (nb == 0) {
        for (int i = threadIdx.x; i < rows * c.d; i += kThreads) static_cast<uint16_t*>(p.o)[row0 * c.d + i] = 0;
        if (threadIdx.x < rows) p.lse[row0 + threadIdx.x] = -INFINITY;
        return;
    }
    const Split split = split_of(total, max_ctas);
    const int64_t u0 = before + item * nb, u1 = u0 + nb;
    const int64_t c0 = split.owner(u0), c1 = split.owner(u1 - 1);
    if (c0 == c1) return;
    for (int i = threadIdx.x; i < rows * (D / 2); i += kThreads) {
        const int r = i / (D / 2), d = i % (D / 2) * 2;
        float big = -INFINITY;
        for (int64_t k = c0; k <= c1; ++k)  // CTA c0's last item, the others' first (c0 too if it began here)
            big = fmaxf(big, partial<D>(p.workspace, k, split.begin(k) >= u0 ? 0 : 1)[kRows * D + 2 * r]);
        const float ref = big == -INFINITY ? 0.f : big;
        float a0 = 0.f, a1 = 0.f, sum = 0.f;
        for (int64_t k = c0; k <= c1; ++k) {
            const float* part = partial<D>(p.workspace, k, split.begin(k) >= u0 ? 0 : 1);
            const float2 ml = *reinterpret_cast<const float2*>(part + kRows * D + 2 * r);
            const float2 v = *reinterpret_cast<const float2*>(part + r * D + d);
            const float f = ex2_approx(ml.x - ref);
            a0 += f * v.x;
            a1 += f * v.y;
            sum += f * ml.y;
        }
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        if (d < c.d)
            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + (row0 + r) * c.d + d) = pack2<kBf16>(a0 * inv, a1 * inv);
        if (d == 0) p.lse[row0 + r] = sum == 0.f ? -INFINITY : (big + lg2_approx(sum)) * kLn2;
    }
}

template <int D, bool kBf16, bool kE4m3>
cudaError_t launch_d(const DecodeParams& p, cudaStream_t stream, int slot) {
    using C = Cfg<D, kE4m3>;
    auto kern = fa2_decode_kernel<D, kBf16, kE4m3>;
    cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), C::kSmem, slot);
    if (e != cudaSuccess) return e;
    kern<<<kMaxCtas, kThreads, C::kSmem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int group = p.heads / p.c.hkv;
    const dim3 grid((unsigned)(p.c.hkv * ((group + kRows - 1) / kRows)), (unsigned)p.c.batch);
    fa2_decode_join_kernel<D, kBf16, C::kKeys><<<grid, kThreads, 0, stream>>>(p, kMaxCtas);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_kind(const DecodeParams& p, cudaStream_t stream, int slot) {
    const bool bf = p.c.dtype == kBf16;
    if (p.c.e4m3) return bf ? launch_d<D, true, true>(p, stream, slot) : launch_d<D, false, true>(p, stream, slot + 1);
    return bf ? launch_d<D, true, false>(p, stream, slot + 2) : launch_d<D, false, false>(p, stream, slot + 3);
}

}  // namespace

size_t decode_workspace_bytes(int, int, int d) {
    return (size_t)kMaxCtas * 2 * kRows * (pad_head_dim(d) + 2) * sizeof(float);
}

cudaError_t launch_decode(const DecodeParams& p, cudaStream_t stream) {
    switch (pad_head_dim(p.c.d)) {
        case 32: return launch_kind<32>(p, stream, 52);
        case 64: return launch_kind<64>(p, stream, 56);
        default: return launch_kind<128>(p, stream, 60);
    }
}

}  // namespace fa2
