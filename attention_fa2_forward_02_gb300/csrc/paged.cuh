// paged.cuh - where a token's row lies in a paged cache, and the conversions of its 8-bit form.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace fa2 {

// A sequence's length as the cache's kernels take it: within [0, room].
__device__ __forceinline__ int bounded_len(int len, int64_t room, unsigned int* status) {
    if (len < 0 || len > room) {
        if (status) atomicOr(status, kStatusBadIndex);
        return len < 0 ? 0 : (int)room;
    }
    return len;
}

// pos / page_size without a division (0 <= pos < 2^31; see page_divisor).
__device__ __forceinline__ int page_of(const PagedParams& c, int pos) {
    return (int)((__umulhi(c.page_mul, (uint32_t)pos) + (uint32_t)pos) >> c.page_shift);
}

// Byte offset of token `pos` of the sequence whose block-table row is `row` (head 0), and its
// index among the scale bytes; -1 where the page number is outside the pool.
struct Slot {
    int64_t off;
    int64_t exp;
};
__device__ __forceinline__ Slot slot_of(const PagedParams& c, int page, int slot) {
    if ((uint64_t)(int64_t)page >= (uint64_t)c.num_pages) {
        if (c.status) atomicOr(c.status, kStatusBadIndex);
        return {-1, -1};
    }
    return {page * c.page_stride + slot * c.slot_stride, (int64_t)page * c.hkv * c.page_size + slot};
}

// The sequence and the position of new token t (fa2_kv_append); false: it has none.
__device__ __forceinline__ bool place_of_row(const PagedParams& c, const int32_t* cu_new, int64_t t, int* seq, int64_t* position) {
    int first = (int)t, end = (int)t + 1, b;
    if (cu_new) {
        // the last sequence that begins at or before row t
        int lo = 0, hi = (int)c.batch;  // cu_new[lo] <= t < cu_new[hi], were it ascending
        if (t < cu_new[0] || t >= cu_new[hi]) return false;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu_new[mid] <= t) lo = mid;
            else hi = mid;
        }
        b = lo;
        first = cu_new[b];
        end = cu_new[b + 1];
    } else {
        b = (int)t;
        if (c.lens[b] == 0) return false;
    }
    const int64_t pos = (int64_t)c.lens[b] - end + t;
    if (t < first || t >= end || pos < 0 || pos >= c.room) {
        if (c.status) atomicOr(c.status, kStatusBadIndex);
        return false;
    }
    *seq = b;
    *position = pos;
    return true;
}

// Two packed e4m3 codes -> two halves (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}

// Four packed e4m3 codes -> the halves of codes 0, 1 and of codes 2, 3.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(codes));
}

// Eight packed e2m1 codes -> four pairs of halves, codes 2 i and 2 i + 1 in pair i (exact).
__device__ __forceinline__ void e2m1x8_to_f16x8(uint32_t codes, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(codes));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&x);
}

}  // namespace fa2
