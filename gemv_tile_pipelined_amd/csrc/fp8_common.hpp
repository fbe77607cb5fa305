// fp8_common.hpp -- what the kernels on block-scaled 8-bit operands share.
//
// An 8-bit operand [R, K] holds e4m3 numbers (1 sign, 4 exponent bits of bias
// 7, 3 fraction bits; +-448 is the largest, 0x7f / 0xff are NaN, there are no
// infinities) and one FP32 scale for each block of `rows` x 128 of them
// (scales [ceil(R / rows), ceil(K / 128)], rows = 1 or 128).
//
// A block's 128 products are added in one of two ways; its sum is then scaled
// and accumulated in FP32.
//  * stream.hip, which waits for memory: the numbers are widened to half
//    precision, which holds every e4m3 number, and multiplied by the 16-bit
//    MFMAs, which add in FP32.  With 8-bit and with 16-bit MFMAs: 1x4096x14336
//    10.8 and 10.9 us, 4x4096x4096 5.1 and 5.3, 4x28672x4096 22.7 and 23.4, 256
//    rows in 64 groups x 2048 x 4096 97.6 and 97.0.
//  * deep.hip and fp8_gemm.hip: the 8-bit MFMAs, at twice the 16-bit ones' rate
//    and with nothing to widen (4096^3 in 16 bits takes 97 us, in fp8_gemm.hip 58
//    to 61; deep.hip took 12.4 us with them and 15.9 with widened numbers for
//    16x4096x14336, 11.3 and 14.7 for 256x4096x4096).  They multiply exactly,
//    but add products in a window aligned to the largest: beside 448 x 448,
//    neighbouring products of 4 and less were lost and of 16 kept (2^-15.6 and
//    2^-13.6 of it).  A sum over 128 came out within 2^-11 of its largest product
//    (measured on normal and on uniformly random bit patterns, all three FP8 MFMA
//    shapes alike; 2^-16 relative to the result in the mean, where rounding a
//    result to bf16 loses up to 2^-8 and to e4m3 2^-4).
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

// a . b + c over 128 e4m3 numbers of each of 16 rows of a and of b, added as an
// 8-bit MFMA adds (the form with no operand scales).
__device__ inline float4_t mfma_fp8(int8_v a, int8_v b, float4_t c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// The 32 bytes of an MFMA operand as 4 operands of 8 half-precision numbers.
struct WideOperand {
  half8_t part[4];
};
__device__ inline WideOperand widen_fp8(int8_v v) {
  WideOperand w;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t four = static_cast<uint32_t>(v[i]);
    const half2_t lo = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(four, 1.0f, false));
    const half2_t hi = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(four, 1.0f, true));
    half8_t &part = w.part[i / 2];
    const int at = i % 2 * 4;
    part[at] = lo[0];
    part[at + 1] = lo[1];
    part[at + 2] = hi[0];
    part[at + 3] = hi[1];
  }
  return w;
}

// a . b over 128 widened numbers, added in FP32: in one chain of MFMAs, or in
// two, which take half as long one after another where a wave has no other MFMAs
// to run meanwhile.
template <int CHAINS>
__device__ inline float4_t mfma_wide(const WideOperand &a, const WideOperand &b) {
  static_assert(CHAINS == 1 || CHAINS == 2, "4 MFMAs");
  float4_t c[CHAINS];
#pragma unroll
  for (int i = 0; i < CHAINS; ++i) c[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i % CHAINS] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.part[i], b.part[i], c[i % CHAINS], 0, 0, 0);
  if constexpr (CHAINS == 2) c[0] += c[1];
  return c[0];
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
