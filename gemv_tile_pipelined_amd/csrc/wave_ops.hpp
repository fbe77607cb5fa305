// wave_ops.hpp -- sums and maxima over a wave's lanes, and 8 packed 16-bit
// numbers as FP32, for the kernels around the products (norm, route, rows).
#pragma once

#include "device_common.hpp"

namespace gt {

typedef uint32_t uint2_v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4_v __attribute__((ext_vector_type(4)));

// v and what the lane sees of it through a DPP lane pattern (0 in lane rows outside
// ROW_MASK), added, or the larger.
template <int CTRL, int ROW_MASK = 0xF>
__device__ inline float dpp_add(float v) {
  const int moved = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROW_MASK, 0xF, false);
  return v + __builtin_bit_cast(float, moved);
}
template <int CTRL, int ROW_MASK = 0xF>
__device__ inline uint32_t dpp_max(uint32_t v) {
  const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROW_MASK, 0xF, false));
  return o > v ? o : v;
}

// Maximum over 8 lanes and over each lane row of 16: pairs, quads, the mirrored half
// row, the mirrored row.
__device__ inline uint32_t max_of_8_lanes(uint32_t v) {
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  return dpp_max<0x141>(v);
}
__device__ inline uint32_t max_of_16_lanes(uint32_t v) { return dpp_max<0x140>(max_of_8_lanes(v)); }

// Sum and maximum over the 64 lanes, in every lane: as above within lane rows,
// then row_bcast:15 adds row 0 into 1 and 2 into 3, row_bcast:31 lane 31 into the
// upper half, and lane 63 has it all.  The order of additions is fixed.
__device__ inline float wave_sum(float v) {
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  v = dpp_add<0x141>(v);
  v = dpp_add<0x140>(v);
  v = dpp_add<0x142, 0xA>(v);
  v = dpp_add<0x143, 0xC>(v);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
template <int CTRL, int ROW_MASK = 0xF>
__device__ inline double dpp_add(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const int low = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROW_MASK, 0xF, false);
  const int high = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROW_MASK, 0xF, false);
  return v + __builtin_bit_cast(double, static_cast<uint64_t>(static_cast<uint32_t>(high)) << 32 | static_cast<uint32_t>(low));
}
// In lane 63 only.
__device__ inline double wave_sum_last(double v) {
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  v = dpp_add<0x141>(v);
  v = dpp_add<0x140>(v);
  v = dpp_add<0x142, 0xA>(v);
  return dpp_add<0x143, 0xC>(v);
}
// Sums over each LANES lanes that follow one another (8 to 64), in every one of them.
template <int LANES>
__device__ inline float lanes_sum(float v) {
  if constexpr (LANES == 64) return wave_sum(v);
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  v = dpp_add<0x141>(v);
  if constexpr (LANES >= 16) v = dpp_add<0x140>(v);
  if constexpr (LANES == 32) v += __shfl_xor(v, 16);
  return v;
}
template <int LANES>
__device__ inline double lanes_sum(double v) {
  if constexpr (LANES == 64) return __shfl(wave_sum_last(v), 63);
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  v = dpp_add<0x141>(v);
  if constexpr (LANES >= 16) v = dpp_add<0x140>(v);
  if constexpr (LANES == 32) v += __shfl_xor(v, 16);
  return v;
}
__device__ inline uint32_t wave_max(uint32_t v) {
  v = max_of_16_lanes(v);
  v = dpp_max<0x142, 0xA>(v);
  v = dpp_max<0x143, 0xC>(v);
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

template <int DT>
__device__ inline void widen8(uint4_v v, float *out) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[2 * i] = widen_in<DT>(static_cast<uint16_t>(v[i]));
    out[2 * i + 1] = widen_in<DT>(static_cast<uint16_t>(v[i] >> 16));
  }
}
template <int DT>
__device__ inline uint4_v round8(const float *v) {
  uint4_v out;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = static_cast<uint32_t>(__builtin_bit_cast(uint16_t, round_out<DT>(v[2 * i]))) |
             static_cast<uint32_t>(__builtin_bit_cast(uint16_t, round_out<DT>(v[2 * i + 1]))) << 16;
  return out;
}

}  // namespace gt
