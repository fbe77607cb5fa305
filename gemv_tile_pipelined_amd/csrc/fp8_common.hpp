// fp8_common.hpp -- what the kernels on block-scaled 8-bit operands share.
//
// An 8-bit operand [R, K] holds e4m3 numbers (1 sign, 4 exponent bits of bias
// 7, 3 fraction bits; +-448 is the largest, 0x7f / 0xff are NaN, there are no
// infinities) and one FP32 scale for each block of `rows` x 128 of them
// (scales [ceil(R / rows), ceil(K / 128)], rows = 1 or 128).
//
// The matrix cores multiply e4m3 numbers exactly and add a step's products in
// a window aligned to the largest one: a sum over 128 products came out within
// 2^-11 of its largest product (measured on normal and on uniformly random bit
// patterns, all three FP8 MFMA shapes alike; 2^-16 relative to the result in
// the mean).  Each 128-wide block's sum is then scaled and accumulated in
// FP32.
#pragma once

#include "device_common.hpp"

namespace gt {

// Columns of K that share a scale; also the K of one v_mfma_*_16x16x128.
constexpr int kScaleBlock = 128;

typedef int int8_v __attribute__((ext_vector_type(8)));

// The 32 bytes of an MFMA operand from two 16-byte pieces.
__device__ inline int8_v join(int4_t lo, int4_t hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// a . b + c over 128 e4m3 numbers of each of 16 rows of a and of b (the form
// with no operand scales).
__device__ inline float4_t mfma_fp8(int8_v a, int8_v b, float4_t c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// As lds_dma_b128, 4 bytes per lane: lane i's dword goes to lds_base + 4 i.
__device__ inline void lds_dma_b32(int4_t rsrc, uint32_t voffset, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dword %0, %2, 0 offen lds"
               : : "v"(voffset), "s"(lds_base), "s"(rsrc) : "memory", "m0");
}
#pragma clang diagnostic pop

}  // namespace gt
