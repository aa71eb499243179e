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
// workspace, at most two per CTA, and the second kernel joins them in CTA order. Two CTAs of
// four warps an SM: one streams while the other ends an item.
//
// The 8-bit cache: with key scale 2^a and value scale 2^e per row, the score of a key is
// x = scale log2(e) 2^a (q . codes) + e, its weight P = 2^(x - m) with m a maximum of x: the
// value's scale is inside the weight, the second product runs on bare codes, and
// l = sum P 2^-e counts the softmax's own terms. Codes are exact in half; q (bfloat16) is
// brought to half exactly by a power of two of its row's largest element.
#include <algorithm>

#include "paged.cuh"

namespace fa2 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;         // query heads per item
constexpr int kMaxCtas = 2 * 152; // CTAs of the first kernel (a fixed number: the split depends on the lengths alone)
constexpr int kJoinWarps = 16;
constexpr int kJoinRows = 4;      // rows a CTA of the second kernel joins
constexpr float kRescale = 8.0f;  // the running maximum may lag by this much (base-2 units) before O is rescaled
constexpr float kLn2 = 0.693147180559945309f;

template <int D, bool kE4m3>
struct Cfg {
    static constexpr int kRowBytes = kE4m3 ? D : 2 * D;
    static constexpr int kKeys = kRowBytes >= 256 ? 16 : (kRowBytes == 128 ? 32 : 64);  // keys per block: 8 KB of K and V
    static constexpr int kLooks = (kKeys + 31) / 32;        // keys a lane looks up per block
    static constexpr int kChunks = kRowBytes / 16;          // 16-byte chunks a row
    static constexpr int kTile = kKeys * kRowBytes;         // K or V of a block
    static constexpr int kInfo = kE4m3 ? kKeys * 16 : 128;  // e4m3: a float4 per key; else the keys that count, as bits
    static constexpr int kStage = 2 * kTile + kInfo;
    static constexpr int kMerge = kRows * (D + 4) * 4;      // a warp's O, m, l at the end of an item
    static constexpr int kStages = kStage * 3 * kWarps > 108 * 1024 ? 2 : (kStage * 4 * kWarps > 108 * 1024 ? 3 : 4);
    static constexpr int kWarpBytes = kStages * kStage > kMerge ? kStages * kStage : kMerge;
    static constexpr int kSmem = kWarps * kWarpBytes;
    static_assert(kStages >= 3 && kSmem <= 112 * 1024, "two CTAs an SM");
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
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
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

// How the blocks of all items are divided over the CTAs. Items are ordered by (sequence, head
// block); every sequence has `per_seq` of them, with the same number of blocks.
struct Split {
    int64_t total;  // blocks in all
    int64_t ctas;   // CTAs that have any: at least a block for each of their warps
    __device__ __forceinline__ Split(int64_t n, int max_ctas) : total(n), ctas((n + kWarps - 1) / kWarps) {
        if (ctas > max_ctas) ctas = max_ctas;
    }
    __device__ __forceinline__ int64_t begin(int64_t c) const { return c * total / ctas; }
    // the CTA that block u belongs to: the largest c with begin(c) <= u
    __device__ __forceinline__ int64_t owner(int64_t u) const {
        int64_t c = u * ctas / total;
        while (c + 1 < ctas && begin(c + 1) <= u) ++c;
        return c;
    }
};

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

// Workspace: per CTA two partial results (its first item, if that began before it or ends after
// it; its last item, if that ends after it), each [kRows][D] floats and then [kRows] (m, l);
// behind all of them, per CTA, the item that begins in it and ends in a later CTA.
template <int D>
__device__ __forceinline__ float* partial(float* ws, int64_t cta, int which) {
    return ws + (cta * 2 + which) * (kRows * (D + 2));
}
struct __align__(16) Torn {
    int rows;      // 0: none
    int last_cta;
    int which;     // the first CTA's partial result
    int out_row;   // row of O and LSE
};
template <int D>
__device__ __forceinline__ Torn* torn(float* ws, int64_t cta) {
    return reinterpret_cast<Torn*>(partial<D>(ws, kMaxCtas, 0)) + cta;
}

// Inclusive sums over the CTA's threads in order, and the total of all. `scratch`: kWarps int64,
// to be used again after the next __syncthreads.
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t* scratch, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    if (lane == 31) scratch[warp] = v;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += scratch[w];
        all += scratch[w];
    }
    *total = all;
    return before + v;
}

template <int D, bool kBf16, bool kE4m3>
__global__ void __launch_bounds__(kThreads, 2) fa2_decode_kernel(const DecodeParams p) {
    using C = Cfg<D, kE4m3>;
    constexpr bool kMmaBf16 = kBf16 && !kE4m3;
    constexpr int kKeys = C::kKeys, S = C::kStages, kNt = kKeys / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scratch[2][kWarps];
    __shared__ int64_t start_seq;
    __shared__ int start_b;
    const PagedParams& c = p.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = p.heads / c.hkv, hblocks = (group + kRows - 1) / kRows;
    const int64_t per_seq = (int64_t)c.hkv * hblocks;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the blocks of all sequences, this CTA's share, and the sequence that it begins in
    int64_t total = 0, mine = 0, upto = 0;  // with at most kThreads sequences: thread i holds sequence i
    const bool one_strip = c.batch <= kThreads;
    if (one_strip) {
        if (threadIdx.x < c.batch) mine = blocks_of<kKeys>(range_of(p, threadIdx.x));
        upto = cta_scan(mine, scratch[0], &total);
    } else {
        for (int b = threadIdx.x; b < c.batch; b += kThreads) mine += blocks_of<kKeys>(range_of(p, b));
        cta_scan(mine, scratch[0], &total);
    }
    const Split split(total * per_seq, gridDim.x);
    const bool working = (int64_t)blockIdx.x < split.ctas;
    const int64_t u_begin = working ? split.begin(blockIdx.x) : 0, u_end = working ? split.begin(blockIdx.x + 1) : 0;
    if (working) {
        if (one_strip) {
            if ((upto - mine) * per_seq <= u_begin && u_begin < upto * per_seq) {
                start_b = threadIdx.x;
                start_seq = (upto - mine) * per_seq;
            }
        } else {
            int64_t before = 0;
            for (int b0 = 0; b0 < c.batch; b0 += kThreads) {
                const int64_t v = b0 + (int)threadIdx.x < c.batch ? blocks_of<kKeys>(range_of(p, b0 + threadIdx.x)) : 0;
                __syncthreads();
                int64_t strip;
                const int64_t to = before + cta_scan(v, scratch[1], &strip);
                if ((to - v) * per_seq <= u_begin && u_begin < to * per_seq) {
                    start_b = b0 + threadIdx.x;
                    start_seq = (to - v) * per_seq;
                }
                before += strip;
                if (before * per_seq > u_begin) break;
            }
        }
    }
    // ---- rows without a key, strewn over the CTAs
    for (int b = blockIdx.x; b < c.batch; b += gridDim.x) {
        const Range r = range_of(p, b);
        if (r.len > r.first) continue;
        const int64_t row0 = (int64_t)b * p.heads;
        for (int i = threadIdx.x; i < p.heads * c.d / 8; i += kThreads)
            reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row0 * c.d)[i] = make_uint4(0, 0, 0, 0);
        for (int i = threadIdx.x; i < p.heads; i += kThreads) p.lse[row0 + i] = -INFINITY;
    }
    if (!working) {
        if (threadIdx.x == 0) torn<D>(p.workspace, blockIdx.x)->rows = 0;
        return;
    }
    __syncthreads();
    int b = start_b;
    int64_t u_seq = start_seq;  // first block of sequence b

    uint8_t* my = smem + warp * C::kWarpBytes;
    const uint32_t my_addr = smem_u32(my);
    const int g = lane >> 2, t = lane & 3;  // row (head) and column group in the products' fragments
    bool first_item = true;
    Torn ends_later{0, 0, 0, 0};

    for (int64_t u = u_begin; u < u_end;) {
        // ---- the item that block u lies in, and this CTA's blocks [k0, k1) of it
        Range range = range_of(p, b);
        int nb = blocks_of<kKeys>(range);
        while (u >= u_seq + nb * per_seq) {
            u_seq += nb * per_seq;
            range = range_of(p, ++b);
            nb = blocks_of<kKeys>(range);
        }
        const int item = (int)((u - u_seq) / nb);
        const int64_t u_item = u_seq + (int64_t)item * nb;
        const int hk = item / hblocks, hb = item % hblocks;
        const int k0 = (int)(u - u_item);
        const int k1 = (int)(u_end - u_item < nb ? u_end - u_item : nb);
        const int head0 = hk * group + hb * kRows;               // first query head
        const int rows = min(kRows, group - hb * kRows);         // query heads of the item

        // ---- the ring: this warp's blocks are k0 + warp, k0 + warp + kWarps, ...
        const int n_mine = k1 - k0 > warp ? (k1 - k0 - warp + kWarps - 1) / kWarps : 0;
        const int32_t* table = c.table + b * c.table_stride;
        const char* kbase = c.k + hk * c.head_stride;
        const char* vbase = c.v + hk * c.head_stride;
        // Lane r looks keys r, r + 32 of a block up. The page numbers are read one block ahead of the
        // copies, the scale bytes with the copies and stored for the products one block later.
        auto key_of = [&](int i, int j) {
            return range.first + (k0 + warp + i * kWarps) * kKeys + (kKeys < 32 ? lane % kKeys : lane + 32 * j);
        };
        int pages[S][C::kLooks];  // of the blocks being started up, then [0]: of the next one
        auto look = [&](int i, int (&page)[C::kLooks]) {
#pragma unroll
            for (int j = 0; j < C::kLooks; ++j) {
                const int key = key_of(i, j);
                page[j] = i < n_mine && key < range.len ? table[key / c.page_size] : -1;
            }
        };
        uint32_t ka[C::kLooks], ve[C::kLooks];  // scale bytes of the block loaded last; ve 256: the key does not count
        auto load = [&](int i, const int (&page)[C::kLooks]) {  // fills stage i % S with block i; commits one group
            if (i < n_mine) {
                const uint32_t st = my_addr + (i % S) * C::kStage;
                int64_t off[C::kLooks];
#pragma unroll
                for (int j = 0; j < C::kLooks; ++j) {
                    const int key = key_of(i, j);
                    Slot s{-1, -1};
                    if (key < range.len) s = slot_of(c, page[j], key % c.page_size);
                    off[j] = s.off;
                    if constexpr (kE4m3) {
                        const int64_t e = s.exp + (int64_t)hk * c.page_size;
                        ka[j] = s.off >= 0 ? c.k_exp[e] : 127u;
                        ve[j] = s.off >= 0 ? c.v_exp[e] : 256u;
                    } else {
                        const uint32_t counts = __ballot_sync(0xffffffffu, s.off >= 0);
                        if (lane == 0) *reinterpret_cast<uint32_t*>(my + (i % S) * C::kStage + 2 * C::kTile + 4 * j) = counts;
                    }
                }
                const int chunk = lane % C::kChunks, r0 = lane / C::kChunks;
                const bool in = chunk * 16 < c.d * (kE4m3 ? 1 : 2);
#pragma unroll
                for (int r = 0; r < kKeys; r += 32 / C::kChunks) {
                    const int64_t o = __shfl_sync(0xffffffffu, off[r / 32], (r & 31) + r0);
                    const bool on = o >= 0 && in;
                    const int64_t at = on ? o + chunk * 16 : 0;
                    const uint32_t dst = st + swizzle<C::kChunks>(r + r0, chunk) * 16;
                    cp_async16(dst, kbase + at, on);
                    cp_async16(dst + C::kTile, vbase + at, on);
                }
            }
            cp_async_commit();
        };
        auto store_info = [&](int i) {  // e4m3: what the products need to know of block i's keys
            if constexpr (kE4m3) {
                if (i >= n_mine) return;
#pragma unroll
                for (int j = 0; j < C::kLooks; ++j) {
                    float4 f;
                    f.x = ka[j] ? __uint_as_float(ka[j] << 23) : 0x1p-127f;
                    f.y = ve[j] < 256 ? (float)((int)ve[j] - 127) : -INFINITY;
                    f.z = ve[j] < 254 ? __uint_as_float((254 - ve[j]) << 23) : 0x1p-127f;
                    f.w = 0.f;
                    reinterpret_cast<float4*>(my + (i % S) * C::kStage + 2 * C::kTile)[lane + 32 * j] = f;
                }
            }
        };
#pragma unroll
        for (int i = 0; i < S; ++i) look(i, pages[i]);

        // ---- q as the first product's left operand: rows g and g + 8
        uint32_t qf[D / 16][4];
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
            }
        }
#pragma unroll
        for (int i = 0; i < S - 1; ++i) {
            load(i, pages[i]);
            store_info(i);
        }
        float qscale[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            qscale[half] = p.scale * 1.4426950408889634f;
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
                qscale[half] *= __uint_as_float((uint32_t)(127 + n) << 23);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w = qf[kk][2 * i + half];
                        qf[kk][2 * i + half] = pack2<false>(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
                    }
            }
        }

        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        int (&page_next)[C::kLooks] = pages[S - 1];

        for (int i = 0; i < n_mine; ++i) {
            cp_async_wait<S - 2>();
            if (i > 0) store_info(i + S - 2);
            __syncwarp();
            load(i + S - 1, page_next);
            look(i + S, page_next);
            const uint32_t kt = my_addr + (i % S) * C::kStage, vt = kt + C::kTile;
            const uint8_t* info = my + (i % S) * C::kStage + 2 * C::kTile;
            // ---- scores: kNt column tiles of 8 keys
            float sc[kNt][4];
#pragma unroll
            for (int j = 0; j < kNt; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
            for (int j = 0; j < kNt; j += 2) {
                const int r = 8 * j + (lane & 7) + (lane & 16 ? 8 : 0);
                if constexpr (!kE4m3) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        uint32_t k4[4];  // (keys 0-7, 8-15) x (d 0-7, 8-15 of this step)
                        ldsm4(kt + swizzle<C::kChunks>(r, 2 * kk + ((lane >> 3) & 1)) * 16, k4);
                        mma16816<kMmaBf16>(sc[j], qf[kk], k4[0], k4[1]);
                        mma16816<kMmaBf16>(sc[j + 1], qf[kk], k4[2], k4[3]);
                    }
                } else {
#pragma unroll
                    for (int kk = 0; kk < D / 16; kk += 2) {
                        uint32_t k4[4];  // (keys 0-7, 8-15) x (16 codes, next 16 codes)
                        ldsm4(kt + swizzle<C::kChunks>(r, kk + ((lane >> 3) & 1)) * 16, k4);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            mma16816<false>(sc[j], qf[kk + h], e4m3x2_to_f16x2(k4[h]), e4m3x2_to_f16x2(k4[h] >> 16));
                            mma16816<false>(sc[j + 1], qf[kk + h], e4m3x2_to_f16x2(k4[2 + h]), e4m3x2_to_f16x2(k4[2 + h] >> 16));
                        }
                    }
                }
            }
            // ---- x, the running maximum, P
            float mx[2] = {-INFINITY, -INFINITY};
            float rv[kNt][2];
            if constexpr (kE4m3) {
#pragma unroll
                for (int j = 0; j < kNt; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 f = reinterpret_cast<const float4*>(info)[8 * j + 2 * t + e];
                        rv[j][e] = f.z;
                        sc[j][e] = fmaf(sc[j][e] * f.x, qscale[0], f.y);
                        sc[j][2 + e] = fmaf(sc[j][2 + e] * f.x, qscale[1], f.y);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < kNt; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[j][e] *= qscale[0];
#pragma unroll
                for (int w = 0; w < C::kLooks; ++w) {
                    const uint32_t counts = reinterpret_cast<const uint32_t*>(info)[w];
                    if (counts != 0xffffffffu) {
#pragma unroll
                        for (int j = 4 * w; j < kNt && j < 4 * w + 4; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (!((counts >> (8 * j + 2 * t + e - 32 * w)) & 1u)) sc[j][e] = sc[j][2 + e] = -INFINITY;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kNt; ++j) {
                mx[0] = fmaxf(mx[0], fmaxf(sc[j][0], sc[j][1]));
                mx[1] = fmaxf(mx[1], fmaxf(sc[j][2], sc[j][3]));
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
            const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
            for (int kt2 = 0; kt2 < kKeys / 16; ++kt2) {
                uint32_t pf[4];
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const int j = 2 * kt2 + jj;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[j][e] = ex2_approx(sc[j][e] - ref[e >> 1]);
                        l[e >> 1] += kE4m3 ? sc[j][e] * rv[j][e & 1] : sc[j][e];
                    }
                    pf[2 * jj] = pack2<kMmaBf16>(sc[j][0], sc[j][1]);
                    pf[2 * jj + 1] = pack2<kMmaBf16>(sc[j][2], sc[j][3]);
                }
                // ---- O += P V
                const int r = 16 * kt2 + (lane & 15);
                if constexpr (!kE4m3) {
#pragma unroll
                    for (int n = 0; n < D / 8; n += 2) {
                        uint32_t v4[4];  // (keys 0-7, 8-15) of chunk n, of chunk n + 1
                        ldsm4_t(vt + swizzle<C::kChunks>(r, n + (lane >> 4)) * 16, v4);
                        mma16816<kMmaBf16>(o[n], pf, v4[0], v4[1]);
                        mma16816<kMmaBf16>(o[n + 1], pf, v4[2], v4[3]);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < D / 16; n += 2) {
                        uint32_t v4[4];  // 16-code chunks n, n + 1: keys 2t, 2t+1 (and + 8) x codes 2g, 2g+1
                        ldsm4_t(vt + swizzle<C::kChunks>(r, n + (lane >> 4)) * 16, v4);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a = __byte_perm(v4[2 * h], 0, 0x3120), b8 = __byte_perm(v4[2 * h + 1], 0, 0x3120);
                            mma16816<false>(o[2 * (n + h)], pf, e4m3x2_to_f16x2(a), e4m3x2_to_f16x2(b8));
                            mma16816<false>(o[2 * (n + h) + 1], pf, e4m3x2_to_f16x2(a >> 16), e4m3x2_to_f16x2(b8 >> 16));
                        }
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
        const int which = first_item ? 0 : 1;
        float* part = partial<D>(p.workspace, blockIdx.x, which);
        const int64_t out_row = (int64_t)b * p.heads + head0;
        if (k0 == 0 && !whole) ends_later = {rows, (int)split.owner(u_item + nb - 1), which, (int)out_row};
        for (int i = threadIdx.x; i < rows * (D / 2); i += kThreads) {
            const int r = i / (D / 2), d = i % (D / 2) * 2;
            float big = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                big = fmaxf(big, reinterpret_cast<const float*>(smem + w * C::kWarpBytes)[r * (D + 4) + D]);
            const float from = big == -INFINITY ? 0.f : big;
            float a0 = 0.f, a1 = 0.f, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* row = reinterpret_cast<const float*>(smem + w * C::kWarpBytes) + r * (D + 4);
                const float f = ex2_approx(row[D] - from);
                a0 += f * row[d];
                a1 += f * row[d + 1];
                sum += f * row[D + 1];
            }
            if (whole) {
                const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
                if (d < c.d)
                    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + (out_row + r) * c.d + d) =
                        pack2<kBf16>(a0 * inv, a1 * inv);
                if (d == 0) p.lse[out_row + r] = sum == 0.f ? -INFINITY : (big + lg2_approx(sum)) * kLn2;
            } else {
                *reinterpret_cast<float2*>(part + r * D + d) = make_float2(a0, a1);
                if (d == 0) *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(big, sum);
            }
        }
        __syncthreads();
        first_item = false;
        u = u_item + k1;
    }
    if (threadIdx.x == 0) *torn<D>(p.workspace, blockIdx.x) = ends_later;
}

// Joins the items that several CTAs worked on: CTA (x, y) rows kJoinRows y .. of the item that
// began in CTA x, if it ended in a later one. A quarter of the warps for each row, a warp for
// every fourth partial result, its lanes for the columns.
template <int D, bool kBf16>
__global__ void __launch_bounds__(kJoinWarps * 32) fa2_decode_join_kernel(const DecodeParams p) {
    constexpr int kShare = kJoinWarps / kJoinRows;  // warps per row
    constexpr int kCols = D / 32;                   // columns a lane
    __shared__ float parts[kJoinWarps][D + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int share = warp % kShare, r = blockIdx.y * kJoinRows + warp / kShare;
    // launched while the first kernel still runs: everything it wrote is here after this wait
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Torn item = *torn<D>(p.workspace, blockIdx.x);
    if ((int)blockIdx.y * kJoinRows >= item.rows) return;
    const int first = blockIdx.x, n = item.last_cta - first + 1;
    const bool on = r < item.rows;
    auto part = [&](int k) { return partial<D>(p.workspace, first + k, k == 0 ? item.which : 0); };
    float big = -INFINITY, sum = 0.f, a[kCols] = {};
    if (on) {
        for (int k = lane; k < n; k += 32) big = fmaxf(big, part(k)[kRows * D + 2 * r]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
        const float from = big == -INFINITY ? 0.f : big;
#pragma unroll 4
        for (int k = share; k < n; k += kShare) {
            const float* s = part(k);
            const float2 ml = *reinterpret_cast<const float2*>(s + kRows * D + 2 * r);
            const float f = ex2_approx(ml.x - from);
            sum += f * ml.y;
#pragma unroll
            for (int i = 0; i < kCols; ++i) a[i] += f * s[r * D + lane + 32 * i];
        }
#pragma unroll
        for (int i = 0; i < kCols; ++i) parts[warp][lane + 32 * i] = a[i];
        if (lane == 0) parts[warp][D] = sum;
    }
    __syncthreads();
    if (!on || share != 0) return;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kShare; ++w) sum += parts[warp + w][D];
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    const int64_t row = (int64_t)item.out_row + r;
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
        const int d = lane + 32 * i;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kShare; ++w) v += parts[warp + w][d];
        if (d < p.c.d) {
            if constexpr (kBf16) static_cast<__nv_bfloat16*>(p.o)[row * p.c.d + d] = __float2bfloat16_rn(v * inv);
            else static_cast<__half*>(p.o)[row * p.c.d + d] = __float2half_rn(v * inv);
        }
    }
    if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : (big + lg2_approx(sum)) * kLn2;
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
    const int rows = std::min(kRows, p.heads / p.c.hkv);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxCtas, (unsigned)((rows + kJoinRows - 1) / kJoinRows), 1);
    cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa2_decode_join_kernel<D, kBf16>, p);
}

template <int D>
cudaError_t launch_kind(const DecodeParams& p, cudaStream_t stream, int slot) {
    const bool bf = p.c.dtype == kBf16;
    if (p.c.e4m3) return bf ? launch_d<D, true, true>(p, stream, slot) : launch_d<D, false, true>(p, stream, slot + 1);
    return bf ? launch_d<D, true, false>(p, stream, slot + 2) : launch_d<D, false, false>(p, stream, slot + 3);
}

}  // namespace

size_t decode_workspace_bytes(int, int, int d) {
    return (size_t)kMaxCtas * (2 * kRows * (pad_head_dim(d) + 2) * sizeof(float) + sizeof(Torn));
}

cudaError_t launch_decode(const DecodeParams& p, cudaStream_t stream) {
    switch (pad_head_dim(p.c.d)) {
        case 32: return launch_kind<32>(p, stream, 52);
        case 64: return launch_kind<64>(p, stream, 56);
        default: return launch_kind<128>(p, stream, 60);
    }
}

}  // namespace fa2
