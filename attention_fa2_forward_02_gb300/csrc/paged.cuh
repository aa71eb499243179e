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

}  // namespace fa2
