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
// running maximum, sum and O, and its own ring of stages filled by asynchronous 16-byte copies
// that run ahead of the products, over the ends of items too: while the CTA adds its warps'
// results up in shared memory at the end of an item, the copies for the next one are under way.
// An item that lies in one CTA is then done, the others leave (m, l, O) in the workspace, at
// most two per CTA, and the second kernel joins them in CTA order. An item counts as kOver
// blocks more than it has, the time its end takes: else the CTA that gets a short sequence's
// many heads finishes last.
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
constexpr int kMergeRows = 4;     // rows the warps add up at a time at the end of an item
constexpr int kOver = 8;          // blocks an item counts beyond its own
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
    static constexpr int kInfo = kE4m3 ? kKeys * 8 : 16;    // e4m3: a float2 per key; else the keys that count, as bits
    static constexpr int kStage = 2 * kTile + kInfo;
    static constexpr int kStages = 2;
    static constexpr bool kQRegs = true;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kQ = kRows * D * 2;                // q as the first product takes it
    static constexpr int kPitch = D + 8;                    // floats a row at the end of an item (no bank twice)
    static constexpr int kMerge = kWarps * kMergeRows * kPitch * 4;
    static constexpr int kSmem = kRing + kQ + kMerge + kRows * 4;
    static_assert(kSmem <= 112 * 1024, "two CTAs an SM");
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

// How the units (units_of) of all items are divided over the CTAs. Items are ordered by
// (sequence, head block); every sequence has `per_seq` of them, with the same number of blocks.
struct Split {
    int64_t total;  // units in all
    int64_t ctas;   // CTAs that have any: at least one for each of their warps
    __device__ __forceinline__ Split(int64_t n, int max_ctas) : total(n), ctas((n + kWarps - 1) / kWarps) {
        if (ctas > max_ctas) ctas = max_ctas;
    }
    __device__ __forceinline__ int64_t begin(int64_t c) const { return c * total / ctas; }
    // the CTA that unit u belongs to: the largest c with begin(c) <= u
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
// What an item of `nb` blocks counts in the division of the work.
__device__ __forceinline__ int units_of(int nb) { return nb ? nb + kOver : 0; }

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

template <bool kBf16>
__device__ __forceinline__ void put(void* o, int64_t i, float v) {
    if constexpr (kBf16) static_cast<__nv_bfloat16*>(o)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(o)[i] = __float2half_rn(v);
}

// A CTA's blocks [k0, k1) of one item, and where the item lies.
struct Segment {
    int64_t u_seq;  // first unit of sequence b
    int64_t next;   // first unit behind the item
    Range range;    // of sequence b
    int b, nb;      // its blocks
    int item, k0, k1;
};

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

    // ---- the units of all sequences, this CTA's share, and the sequence that it begins in
    int64_t total = 0, mine = 0, upto = 0;  // with at most kThreads sequences: thread i holds sequence i
    const bool one_strip = c.batch <= kThreads;
    if (one_strip) {
        if (threadIdx.x < c.batch) mine = units_of(blocks_of<kKeys>(range_of(p, threadIdx.x)));
        upto = cta_scan(mine, scratch[0], &total);
    } else {
        for (int b = threadIdx.x; b < c.batch; b += kThreads) mine += units_of(blocks_of<kKeys>(range_of(p, b)));
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
                const int64_t v = b0 + (int)threadIdx.x < c.batch ? units_of(blocks_of<kKeys>(range_of(p, b0 + threadIdx.x))) : 0;
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

    // the segment that unit u lies in; false: the CTA has no block from u on
    auto seek = [&](Segment& s, int64_t u) {
        if (u >= u_end) return false;
        while (u >= s.u_seq + units_of(s.nb) * per_seq) {
            s.u_seq += units_of(s.nb) * per_seq;
            s.range = range_of(p, ++s.b);
            s.nb = blocks_of<kKeys>(s.range);
        }
        const int units = units_of(s.nb);
        s.item = (int)((u - s.u_seq) / units);
        const int64_t u_item = s.u_seq + (int64_t)s.item * units;  // kOver units first, then the blocks
        const int64_t from = u - u_item - kOver, to = u_end - u_item - kOver;
        s.k0 = from > 0 ? (int)from : 0;
        s.k1 = to < s.nb ? (int)to : s.nb;
        s.next = u_item + units;
        return s.k1 > s.k0;
    };
    // this warp's blocks of segment number `number`: k0 + turn(number), + kWarps, ...
    auto turn = [&](int number) { return (warp + number) % kWarps; };
    auto count = [&](const Segment& s, int number) {
        const int n = s.k1 - s.k0 - turn(number);
        return n > 0 ? (n + kWarps - 1) / kWarps : 0;
    };

    Segment seg;
    seg.b = start_b;
    seg.u_seq = start_seq;
    seg.range = range_of(p, seg.b);
    seg.nb = blocks_of<kKeys>(seg.range);
    bool live = seek(seg, u_begin);

    // ---- the ring. Lane r looks keys r, r + 32 of a block up; the page numbers are read one block
    // ahead of the copies (`ahead`), the scale bytes with the copies and stored one block later.
    uint8_t* my = smem + warp * S * C::kStage;
    const uint32_t my_addr = smem_u32(my);
    Segment ahead = seg;
    bool ahead_live = live;
    int ahead_number = 0, ahead_left = 0, ahead_key = 0;  // blocks of this warp left, the next one's first key
    const int32_t* ahead_table = nullptr;
    int64_t ahead_head = 0, ahead_exp = 0;                // the head's offset in a page, in its scale bytes
    auto enter = [&]() {
        if (!ahead_live) return;
        const int hk = ahead.item / hblocks;
        ahead_left = count(ahead, ahead_number);
        ahead_key = ahead.range.first + (ahead.k0 + turn(ahead_number)) * kKeys + (kKeys < 32 ? lane % kKeys : lane);
        ahead_table = c.table + ahead.b * c.table_stride;
        ahead_head = hk * c.head_stride;
        ahead_exp = (int64_t)hk * c.page_size;
    };
    enter();
    int page[C::kLooks], slot[C::kLooks];  // slot -1: no such key
    int64_t head_off = 0, head_exp = 0;    // and the block's head
    bool found = false;
    auto look = [&]() {  // the next block of this warp, if there is one
        while (ahead_live && ahead_left == 0) {
            ahead_live = seek(ahead, ahead.next);
            ++ahead_number;
            enter();
        }
        found = ahead_live;
        if (!found) return;
        head_off = ahead_head;
        head_exp = ahead_exp;
#pragma unroll
        for (int j = 0; j < C::kLooks; ++j) {
            const int key = ahead_key + 32 * j;
            page[j] = 0;
            slot[j] = -1;
            if (key < ahead.range.len) {
                const int at = page_of(c, key);
                page[j] = ahead_table[at];
                slot[j] = key - at * c.page_size;
            }
        }
        ahead_key += kWarps * kKeys;
        --ahead_left;
    };
    int fill = 0;                        // the stage to fill next
    uint32_t ka[C::kLooks], ve[C::kLooks];  // scale bytes of the block loaded last; ve 256: the key does not count
    int info_stage = -1;                 // and its stage, while they are not stored
    auto load = [&]() {  // copies the block looked up last into the next stage; commits one group
        if (found) {
            const uint32_t st = my_addr + fill * C::kStage;
            const char* kbase = c.k + head_off;
            const char* vbase = c.v + head_off;
            int64_t off[C::kLooks];
#pragma unroll
            for (int j = 0; j < C::kLooks; ++j) {
                Slot s{-1, -1};
                if (slot[j] >= 0) s = slot_of(c, page[j], slot[j]);
                off[j] = s.off;
                if constexpr (kE4m3) {
                    const int64_t e = s.exp + head_exp;
                    ka[j] = s.off >= 0 ? c.k_exp[e] : 127u;
                    ve[j] = s.off >= 0 ? c.v_exp[e] : 256u;
                } else {
                    const uint32_t counts = __ballot_sync(0xffffffffu, s.off >= 0);
                    if (lane == 0) *reinterpret_cast<uint32_t*>(my + fill * C::kStage + 2 * C::kTile + 4 * j) = counts;
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
            info_stage = fill;
        }
        cp_async_commit();
        fill = fill + 1 == S ? 0 : fill + 1;
    };
    auto store_info = [&]() {  // e4m3: the key's scale, and the value scale's exponent (-infinity: masked)
        if constexpr (kE4m3) {
            if (info_stage < 0) return;
#pragma unroll
            for (int j = 0; j < C::kLooks; ++j)
                reinterpret_cast<float2*>(my + info_stage * C::kStage + 2 * C::kTile)[lane + 32 * j] =
                    make_float2(__uint_as_float(ka[j] << 23), ve[j] < 256 ? (float)((int)ve[j] - 127) : -INFINITY);
            info_stage = -1;
        }
    };
    look();
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        load();
        look();
        store_info();
    }

    uint8_t* q_smem = smem + C::kRing;
    float* merge = reinterpret_cast<float*>(smem + C::kRing + C::kQ);
    float* q_scale = reinterpret_cast<float*>(smem + C::kRing + C::kQ + C::kMerge);
    const uint32_t q_addr = smem_u32(q_smem), q_off = swizzle<D / 8>((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4) * 16;
    const int g = lane >> 2, t = lane & 3;  // row (head) and column group in the products' fragments
    int number = 0, use = 0;                // the segment's number, the stage to use next
    bool first_item = true;
    Torn ends_later{0, 0, 0, 0};

    for (; live; ++number) {
        const int hk = seg.item / hblocks, hb = seg.item % hblocks;
        const int head0 = hk * group + hb * kRows;        // first query head
        const int rows = min(kRows, group - hb * kRows);  // query heads of the item

        // ---- q into shared memory: thread (row, 16 elements)
        if (threadIdx.x < D) {
            constexpr int kParts = D / 16;
            const int r = threadIdx.x / kParts, part = threadIdx.x % kParts;
            const uint16_t* src = static_cast<const uint16_t*>(p.q) + seg.b * p.q_batch + (int64_t)(head0 + r) * p.q_head + 16 * part;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const uint4 lo = r < rows && 16 * part < c.d ? *reinterpret_cast<const uint4*>(src) : zero;
            const uint4 hi = r < rows && 16 * part + 8 < c.d ? *reinterpret_cast<const uint4*>(src + 8) : zero;
            uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            float scale = p.scale * 1.4426950408889634f;
            if constexpr (kBf16 && kE4m3) {
                float a = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    a = fmaxf(a, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
#pragma unroll
                for (int off = kParts / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
                // 2^n with a 2^-n in [2^14, 2^15): half's range then reaches 2^-38 of the largest element
                int n = (int)(__float_as_uint(a) >> 23) - 127 - 14;
                if (a == 0.f || !(a < INFINITY)) n = 0;
                if (n < -126) n = -126;
                const float up = __uint_as_float((uint32_t)(127 - n) << 23);
                scale *= __uint_as_float((uint32_t)(127 + n) << 23);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = pack2<false>(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
            }
            // 8-bit cache: elements 4t .. 4t+3 of 16 as columns 2t, 2t+1, 2t+8, 2t+9, the order its codes come in
            uint4* row = reinterpret_cast<uint4*>(q_smem);
            row[swizzle<D / 8>(r, 2 * part)] = kE4m3 ? make_uint4(w[0], w[2], w[4], w[6]) : make_uint4(w[0], w[1], w[2], w[3]);
            row[swizzle<D / 8>(r, 2 * part + 1)] = kE4m3 ? make_uint4(w[1], w[3], w[5], w[7]) : make_uint4(w[4], w[5], w[6], w[7]);
            if (part == 0) q_scale[r] = scale;
        }
        __syncthreads();
        const float qscale[2] = {q_scale[g], q_scale[g + 8]};
        uint32_t qf[C::kQRegs ? D / 16 : 1][4];
        if constexpr (C::kQRegs) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) ldsm4(q_addr + (q_off ^ (uint32_t)(2 * kk * 16)), qf[kk]);
        }

        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (int i = count(seg, number); i > 0; --i) {
            cp_async_wait<S - 2>();
            store_info();
            __syncwarp();
            load();
            look();
            const uint32_t kt = my_addr + use * C::kStage, vt = kt + C::kTile;
            const uint8_t* info = my + use * C::kStage + 2 * C::kTile;
            use = use + 1 == S ? 0 : use + 1;
            // ---- scores: kNt column tiles of 8 keys
            float sc[kNt][4];
#pragma unroll
            for (int j = 0; j < kNt; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
            const int kr = (lane & 7) + (lane & 16 ? 8 : 0);
#pragma unroll
            for (int kk = 0; kk < D / 16; kk += 2) {
                uint32_t qa[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (C::kQRegs) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) qa[h][i] = qf[kk + h][i];
                    } else {  // the swizzle's exclusive or commutes with the constant chunk offset
                        ldsm4(q_addr + (q_off ^ (uint32_t)(2 * (kk + h) * 16)), qa[h]);
                    }
                }
#pragma unroll
                for (int j = 0; j < kNt; j += 2) {
                    if constexpr (!kE4m3) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t k4[4];  // (keys 0-7, 8-15) x (d 0-7, 8-15 of this step)
                            ldsm4(kt + swizzle<C::kChunks>(8 * j + kr, 2 * (kk + h) + ((lane >> 3) & 1)) * 16, k4);
                            mma16816<kMmaBf16>(sc[j], qa[h], k4[0], k4[1]);
                            mma16816<kMmaBf16>(sc[j + 1], qa[h], k4[2], k4[3]);
                        }
                    } else {
                        uint32_t k4[4];  // (keys 0-7, 8-15) x (16 codes, next 16 codes)
                        ldsm4(kt + swizzle<C::kChunks>(8 * j + kr, kk + ((lane >> 3) & 1)) * 16, k4);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t b0, b1, b2, b3;
                            e4m3x4_to_f16x4(k4[h], b0, b1);
                            e4m3x4_to_f16x4(k4[2 + h], b2, b3);
                            mma16816<false>(sc[j], qa[h], b0, b1);
                            mma16816<false>(sc[j + 1], qa[h], b2, b3);
                        }
                    }
                }
            }
            // ---- x, the running maximum, P
            float mx[2] = {-INFINITY, -INFINITY};
            float rv[kNt][2];
            if constexpr (kE4m3) {
#pragma unroll
                for (int j = 0; j < kNt; ++j) {
                    const float4 f = reinterpret_cast<const float4*>(info)[4 * j + t];  // keys 8 j + 2 t, + 1
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float ks = e ? f.z : f.x, ex = e ? f.w : f.y;
                        // 2^-ex out of the low bits of 1.5 2^23 + 127 - ex; masked: 0
                        rv[j][e] = __uint_as_float(__float_as_uint(12583039.f - ex) << 23);
                        sc[j][e] = fmaf(sc[j][e] * ks, qscale[0], ex);
                        sc[j][2 + e] = fmaf(sc[j][2 + e] * ks, qscale[1], ex);
                    }
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
                            uint32_t b0, b1, b2, b3;  // keys 2t, 2t+1 of the even, of the odd code; keys + 8
                            e4m3x4_to_f16x4(__byte_perm(v4[2 * h], 0, 0x3120), b0, b2);
                            e4m3x4_to_f16x4(__byte_perm(v4[2 * h + 1], 0, 0x3120), b1, b3);
                            mma16816<false>(o[2 * (n + h)], pf, b0, b1);
                            mma16816<false>(o[2 * (n + h) + 1], pf, b2, b3);
                        }
                    }
                }
            }
            __syncwarp();  // the stage may be filled again
        }

        // ---- the warps' results together, kMergeRows rows at a time: a warp per row, a lane per D / 32 columns
        const bool whole = seg.k0 == 0 && seg.k1 == seg.nb;
        const int which = first_item ? 0 : 1;
        const int64_t out_row = (int64_t)seg.b * p.heads + head0;
        if (seg.k0 == 0 && !whole) ends_later = {rows, (int)split.owner(seg.next - 1), which, (int)out_row};
        float* part = partial<D>(p.workspace, blockIdx.x, which);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
#pragma unroll
        for (int round = 0; round < kRows / kMergeRows; ++round) {
            if (round * kMergeRows >= rows) break;
            const int h = round / 2;
            if (g / kMergeRows == round % 2) {
                float* row = merge + (warp * kMergeRows + g % kMergeRows) * C::kPitch;
#pragma unroll
                for (int n = 0; n < D / 8; n += 2) {
                    if constexpr (!kE4m3) {  // columns 8 n + 2 t, + 1
                        *reinterpret_cast<float2*>(row + 8 * n + 2 * t) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
                        *reinterpret_cast<float2*>(row + 8 * n + 8 + 2 * t) = make_float2(o[n + 1][2 * h], o[n + 1][2 * h + 1]);
                    } else {  // tiles n, n + 1 hold the even and odd codes of a chunk: columns 8 n + 4 t .. + 3
                        *reinterpret_cast<float4*>(row + 8 * n + 4 * t) =
                            make_float4(o[n][2 * h], o[n + 1][2 * h], o[n][2 * h + 1], o[n + 1][2 * h + 1]);
                    }
                }
                if (t == 0) *reinterpret_cast<float2*>(row + D) = make_float2(m[h], l[h]);
            }
            __syncthreads();
            const int r = round * kMergeRows + warp;
            if (r < rows) {
                constexpr int kCols = D / 32;
                float big = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) big = fmaxf(big, merge[(w * kMergeRows + warp) * C::kPitch + D]);
                const float from = big == -INFINITY ? 0.f : big;
                float a[kCols] = {}, sum = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float* row = merge + (w * kMergeRows + warp) * C::kPitch;
                    const float f = ex2_approx(row[D] - from);
                    sum += f * row[D + 1];
#pragma unroll
                    for (int i = 0; i < kCols; ++i) a[i] += f * row[lane + 32 * i];
                }
                if (whole) {
                    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
                        if (lane + 32 * i < c.d) put<kBf16>(p.o, (out_row + r) * c.d + lane + 32 * i, a[i] * inv);
                    if (lane == 0) p.lse[out_row + r] = sum == 0.f ? -INFINITY : (big + lg2_approx(sum)) * kLn2;
                } else {
#pragma unroll
                    for (int i = 0; i < kCols; ++i) part[r * D + lane + 32 * i] = a[i];
                    if (lane == 0) *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(big, sum);
                }
            }
            __syncthreads();
        }
        first_item = false;
        live = seek(seg, seg.next);
    }
    cp_async_wait<0>();
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
        if (d < p.c.d) put<kBf16>(p.o, row * p.c.d + d, v * inv);
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
