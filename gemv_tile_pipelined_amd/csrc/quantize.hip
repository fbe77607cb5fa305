// quantize.hip -- 16-bit numbers to e4m3 with an FP32 scale for each block of
// 1 x 128 (activations) or 128 x 128 (weights) of them.
//
//   scale = max(amax / 448, 2^-80)      amax = largest |x| of the block
//   q     = the e4m3 number nearest to the real quotient x / scale, ties to even
//
// scale is the correctly rounded FP32 quotient.  The floor keeps the scale of
// a block of zeros (or of values below 448 * 2^-80) a normal number whose
// residuals below stay representable.  A NaN or an infinity in a block makes its
// scale NaN or infinite, so that everything multiplied with the block is NaN
// (over an infinite scale finite numbers are zeros and infinities NaN).
//
// The nearest e4m3 number of the real quotient, not of its FP32 rounding: the
// FP32 quotient may land exactly between two e4m3 numbers when the real one
// does not.  The quotient is therefore rounded to odd first (truncated, with the
// last bit set if anything was cut off), which leaves the tie to the
// conversion only if it is one.  The residual fma(-q, scale, x) is exact up
// to its own rounding and so has the right sign; one Newton step brings q
// within one unit in the last place of the real quotient, which is all that
// the truncation needs.
//
// Bound by memory: 2 bytes read and 1 written per element, each once; a
// block's elements stay in registers between the maximum and the rounding.
// 8192 x 4096 by rows 19 us, 5.4 TB/s (a copy of a large tensor: 5.1); 4095 x
// 14336 in tiles 34.5 us, 5.1 TB/s.
#include "fp8_common.hpp"
#include "groups.hpp"
#include "kernels.hpp"

namespace gt {

namespace {

typedef unsigned short ushort2_v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4_v __attribute__((ext_vector_type(4)));

constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 0x1p-80f;

// Largest |x| of 8 packed 16-bit numbers, as bits: without the sign bit, both
// formats order like unsigned integers, NaN above infinity above the rest.
__device__ inline uint32_t abs_max16(uint32_t m, uint4_v v) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2_v, m),
                                                               __builtin_bit_cast(ushort2_v, v[i] & 0x7fff7fffu)));
  return m;
}

__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Larger of this lane's value and that of a lane of the same row of 16,
// chosen by a DPP control.
template <int CTRL>
__device__ inline uint32_t dpp_max(uint32_t v) {
  return umax(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, false)));
}
// Maximum over each aligned group of 8 lanes: pairs, quads (quad_perm), then
// the mirrored half row.
__device__ inline uint32_t max_of_8_lanes(uint32_t v) {
  v = dpp_max<0xB1>(v);   // quad_perm [1,0,3,2]
  v = dpp_max<0x4E>(v);   // quad_perm [2,3,0,1]
  return dpp_max<0x141>(v);  // row_half_mirror
}

template <int DT>
__device__ inline float block_scale(uint32_t amax_bits) {
  const float s = widen_in<DT>(static_cast<uint16_t>(amax_bits)) / kE4m3Max;
  return s < kMinScale ? kMinScale : s;  // a NaN stays
}

// What quotient_to_odd divides by.  An infinite scale (inv = 0) would make its
// residuals NaN: beside any finite divisor finite x come out below the smallest
// e4m3 number, and infinite ones NaN.
__device__ inline float divisor(float scale) { return scale == __builtin_inff() ? 0x1.fffffep127f : scale; }

// x / scale rounded to odd (see the top of the file); inv is about 1 / scale.
__device__ inline float quotient_to_odd(float x, float scale, float inv) {
  const float a = __builtin_fabsf(x);
  float q = a * inv;
  q = __builtin_fmaf(__builtin_fmaf(-q, scale, a), inv, q);
  const float r = __builtin_fmaf(-q, scale, a);
  uint32_t b = __builtin_bit_cast(uint32_t, q);
  b -= r < 0.0f ? 1u : 0u;
  b |= r != 0.0f ? 1u : 0u;
  return __builtin_copysignf(__builtin_bit_cast(float, b), x);
}

// 4 packed 16-bit numbers to 4 e4m3 numbers.
template <int DT>
__device__ inline uint32_t quantize4(uint32_t lo, uint32_t hi, float scale, float inv) {
  const float a = quotient_to_odd(widen_in<DT>(static_cast<uint16_t>(lo)), scale, inv);
  const float b = quotient_to_odd(widen_in<DT>(static_cast<uint16_t>(lo >> 16)), scale, inv);
  const float c = quotient_to_odd(widen_in<DT>(static_cast<uint16_t>(hi)), scale, inv);
  const float d = quotient_to_odd(widen_in<DT>(static_cast<uint16_t>(hi >> 16)), scale, inv);
  const int half = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, half, true));
}

template <int DT>
__device__ inline uint4_v quantize16(uint4_v v0, uint4_v v1, float scale, float inv) {
  uint4_v q;
  q[0] = quantize4<DT>(v0[0], v0[1], scale, inv);
  q[1] = quantize4<DT>(v0[2], v0[3], scale, inv);
  q[2] = quantize4<DT>(v1[0], v1[1], scale, inv);
  q[3] = quantize4<DT>(v1[2], v1[3], scale, inv);
  return q;
}

// Row blocks: 8 lanes hold a block's 128 columns, 16 each (one 16-byte store;
// K % 16 == 0, so a lane's columns are all inside the row or all outside).
// A wave's 8 blocks follow one another along the row and then down the rows.
// q stays cached: non-temporal stores take 1.5 us off 8192 x 4096 alone (21.4 ->
// 19.8), but the product that reads q next then takes 3 us longer.
constexpr int kRowThreads = 256;
constexpr int kRowBlocks = kRowThreads / 8;
template <int DT>
__global__ void __launch_bounds__(kRowThreads)
quantize_rows_kernel(const uint16_t *__restrict__ x, uint8_t *__restrict__ q, float *__restrict__ scale, uint32_t blocks,
                     uint32_t per_row, int K) {
  // Fewer than 2^29 blocks (the library's limit): 32-bit numbers.
  const uint32_t b = blockIdx.x * kRowBlocks + (threadIdx.x >> 3);
  if (b >= blocks) return;  // all 8 lanes of a block alike
  const uint32_t row = b / per_row;
  const int k = static_cast<int>(b - row * per_row) * kScaleBlock + static_cast<int>(threadIdx.x & 7) * 16;
  const int64_t at = static_cast<int64_t>(row) * K + k;
  uint4_v v0 = {0, 0, 0, 0}, v1 = {0, 0, 0, 0};
  if (k < K) {
    v0 = *reinterpret_cast<const uint4_v *>(x + at);
    v1 = *reinterpret_cast<const uint4_v *>(x + at + 8);
  }
  uint32_t m = abs_max16(abs_max16(0, v0), v1);
  m = max_of_8_lanes(umax(m & 0xffffu, m >> 16));
  const float s = block_scale<DT>(m);
  if ((threadIdx.x & 7) == 0) scale[b] = s;
  if (k < K) *reinterpret_cast<uint4_v *>(q + at) = quantize16<DT>(v0, v1, divisor(s), 1.0f / s);
}

// Whether the tiles' q leaves with non-temporal stores: when what is read and
// written does not fit the L2s (32 MiB), so that a later reader would not find it
// there anyway.  Cached and non-temporal: 4096 x 4096 12.1 and 10.7 us, 14336 x
// 4096 35.0 and 33.7, 1000 x 1040 4.1 and 4.5.
bool streamed(int64_t elements) { return elements > (int64_t{1} << 25) / 3; }

// Tiles: a workgroup holds a 128 x 128 tile, 8 lanes to a row, 64 rows at a
// time (4095 x 14336: 256 threads, 32 rows at a time, 40.7 us, 512 threads 36.5,
// 1024 threads 46).
constexpr int kTileThreads = 512;
template <int DT>
__global__ void __launch_bounds__(kTileThreads)
quantize_tiles_kernel(const uint16_t *__restrict__ x, uint8_t *__restrict__ q, float *__restrict__ scale, int N, int K,
                      int tiles_n, int tiles_k, bool past_l2) {
  __shared__ uint32_t wave_max[kTileThreads / 64];
  constexpr int kPasses = kScaleBlock * 8 / kTileThreads;
  const unsigned per = static_cast<unsigned>(tiles_n) * static_cast<unsigned>(tiles_k);
  const unsigned e = blockIdx.x / per, t = blockIdx.x % per;
  const int n0 = static_cast<int>(t / static_cast<unsigned>(tiles_k)) * kScaleBlock;
  const int k = static_cast<int>(t % static_cast<unsigned>(tiles_k)) * kScaleBlock + (threadIdx.x & 7) * 16;
  const int64_t base = static_cast<int64_t>(e) * N * K + k;
  uint4_v v[kPasses][2];
  uint32_t m = 0;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int n = n0 + p * (kTileThreads / 8) + (threadIdx.x >> 3);
    v[p][0] = v[p][1] = uint4_v{0, 0, 0, 0};
    if (n < N && k < K) {
      const uint16_t *src = x + base + static_cast<int64_t>(n) * K;
      v[p][0] = *reinterpret_cast<const uint4_v *>(src);
      v[p][1] = *reinterpret_cast<const uint4_v *>(src + 8);
    }
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) m = abs_max16(abs_max16(m, v[p][0]), v[p][1]);
  m = max_of_8_lanes(umax(m & 0xffffu, m >> 16));
#pragma unroll
  for (int lane = 8; lane < 64; lane <<= 1) m = umax(m, __shfl_xor(m, lane));
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTileThreads / 64; ++w) m = umax(m, wave_max[w]);
  const float s = block_scale<DT>(m);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
  const float d = divisor(s), inv = 1.0f / s;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int n = n0 + p * (kTileThreads / 8) + (threadIdx.x >> 3);
    if (n < N && k < K) {
      const uint4_v out = quantize16<DT>(v[p][0], v[p][1], d, inv);
      uint4_v *const dst = reinterpret_cast<uint4_v *>(q + base + static_cast<int64_t>(n) * K);
      if (past_l2)
        __builtin_nontemporal_store(out, dst);
      else
        *dst = out;
    }
  }
}

}  // namespace

hipError_t launch_quantize_rows(int dtype, const void *x, void *q, float *scale, int64_t M, int K, hipStream_t stream) {
  const int per_row = (K + kScaleBlock - 1) / kScaleBlock;
  const int64_t blocks = M * per_row;
  const dim3 grid(static_cast<unsigned>((blocks + kRowBlocks - 1) / kRowBlocks));
  const auto kernel = dtype == kBF16 ? quantize_rows_kernel<kBF16> : quantize_rows_kernel<kF16>;
  hipLaunchKernelGGL(kernel, grid, dim3(kRowThreads), 0, stream, static_cast<const uint16_t *>(x),
                     static_cast<uint8_t *>(q), scale, static_cast<uint32_t>(blocks), static_cast<uint32_t>(per_row), K);
  return hipGetLastError();
}

hipError_t launch_quantize_tiles(int dtype, const void *x, void *q, float *scale, int E, int N, int K,
                                 hipStream_t stream) {
  const int tiles_n = (N + kScaleBlock - 1) / kScaleBlock, tiles_k = (K + kScaleBlock - 1) / kScaleBlock;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(E) * tiles_n * tiles_k));
  const auto kernel = dtype == kBF16 ? quantize_tiles_kernel<kBF16> : quantize_tiles_kernel<kF16>;
  hipLaunchKernelGGL(kernel, grid, dim3(kTileThreads), 0, stream, static_cast<const uint16_t *>(x),
                     static_cast<uint8_t *>(q), scale, N, K, tiles_n, tiles_k,
                     streamed(static_cast<int64_t>(E) * N * K));
  return hipGetLastError();
}

}  // namespace gt
