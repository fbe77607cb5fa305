// fp4.hip -- weights in 4 bits: the product of a few rows with them, and the
// quantiser that makes them.
//
// A 4-bit operand [N, K] holds e2m1 numbers (1 sign, 2 exponent bits of bias 1,
// 1 fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte with the even
// column in the low half, and one scale byte s for each 32 of a row, which
// stands for 2^(s - 127) (255: NaN).
//
//   y[m,n] = sum_b 2^(s[n,b] - 127) * sum_{k in block b} x[m,k] * W[n,k]
//
// The product reads 17 bytes of W for 32 numbers, each once, and is bound by
// that.  One v_cvt_scalef32_pk_*_fp4 turns a byte into two numbers of x's
// format, which holds every e2m1 number, so a product of 16-bit MFMAs
// (16x16x32) adds exact products in FP32; a block's sum is then scaled in FP32,
// which is exact but for results below FP32's normal numbers.  (Scaled in the
// conversion instead, half precision would overflow or lose bits of small
// blocks.)
//
// Lane n + 16 g of a wave loads 16 bytes of row n: the whole block g of four
// blocks that follow one another.  An MFMA wants all four lane rows to hold 8
// numbers each of one block, which is the transpose of 4 x 4 dwords across lane
// rows: two v_permlane32_swap and two v_permlane16_swap.
#include "device_common.hpp"
#include "kernels.hpp"
#include "wave_ops.hpp"

namespace gt {

namespace {

typedef unsigned short ushort2_v __attribute__((ext_vector_type(2)));

constexpr int kFp4Block = 32;   // numbers that share a scale; also the K of one MFMA
constexpr int kFp4Chunk = 128;  // columns that a wave takes at a time

// The 8 numbers of a dword in x's format.
template <int DT>
__device__ inline half8_t widen_fp4(uint32_t v) {
  half8_t w;
  if constexpr (DT == kF16) {
    const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 0);
    const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 1);
    const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 2);
    const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 3);
    w = half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 0);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 1);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 2);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 3);
    w = __builtin_bit_cast(half8_t, bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]});
  }
  return w;
}

template <int DT>
__device__ inline float4_t mfma_16x16x32(half8_t a, half8_t b) {
  const float4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (DT == kF16) return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, zero, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), zero, 0, 0, 0);
}

// 4 x 4 dwords across the four lane rows: v[i] of lane row g <-> v[g] of row i.
__device__ inline uint4_v transpose_rows(uint4_v v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return uint4_v{c[0], c[1], d[0], d[1]};
}

// 2^(s - 127) of byte i: the byte as an FP32 exponent, but for 0 (2^-127, below
// the normal numbers) and 255 (NaN).
__device__ inline float scale_of(uint32_t bytes, int i) {
  const uint32_t s = (bytes >> (8 * i)) & 0xffu;
  const uint32_t bits = s << 23;
  const float f = __builtin_bit_cast(float, bits > 0x00400000u ? bits : 0x00400000u);
  return s == 0xffu ? __builtin_nanf("") : f;
}

// A workgroup has NT * 16 rows of W and up to MT * 16 rows of x; its waves take
// the chunks of K in turn and their sums meet in LDS, added in wave order.
// FULL: all 16 rows of each block of x, four sums to a lane; otherwise one row,
// which only the first register of each sum holds.
template <int DT, int MT, int NT, int WAVES, int DEPTH, bool FULL>
__global__ void __launch_bounds__(WAVES * 64)
gemv_fp4_kernel(const uint16_t *__restrict__ x, const uint8_t *__restrict__ W, const uint8_t *__restrict__ sW,
                uint16_t *__restrict__ y, int M, int N, int K) {
  constexpr int R = FULL ? 4 : 1;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int n0 = static_cast<int>(blockIdx.x) * (NT * 16);
  const int m0 = static_cast<int>(blockIdx.y) * (MT * 16);
  // Rows past the last read the last one again; what they give is not stored.
  const uint16_t *xrow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    int m = m0 + t * 16 + i16;
    if (m >= M) m = M - 1;
    xrow[t] = x + static_cast<int64_t>(m) * K + g * 8;
  }
  const uint8_t *wrow[NT], *srow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    int n = n0 + t * 16 + i16;
    if (n >= N) n = N - 1;
    wrow[t] = W + static_cast<int64_t>(n) * (K / 2);
    srow[t] = sW + static_cast<int64_t>(n) * (K / kFp4Block);
  }
  float acc[NT][MT][R];
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int b = 0; b < MT; ++b)
#pragma unroll
      for (int r = 0; r < R; ++r) acc[a][b][r] = 0.0f;

  struct Chunk {
    uint4_v w[NT];
    uint32_t s[NT];
    half8_t x[MT][4];
  };
  auto load = [&](Chunk &c, int chunk) {
    const int64_t k = static_cast<int64_t>(chunk) * kFp4Chunk;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      c.w[t] = *reinterpret_cast<const uint4_v *>(wrow[t] + k / 2 + g * 16);
      __builtin_memcpy(&c.s[t], srow[t] + k / kFp4Block, 4);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) c.x[t][i] = *reinterpret_cast<const half8_t *>(xrow[t] + k + i * kFp4Block);
  };
  auto multiply = [&](const Chunk &c, int blocks) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint4_v w = transpose_rows(c.w[t]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < blocks) {
          const half8_t b = widen_fp4<DT>(w[i]);
          const float s = scale_of(c.s[t], i);
#pragma unroll
          for (int u = 0; u < MT; ++u) {
            const float4_t part = mfma_16x16x32<DT>(c.x[u][i], b);
#pragma unroll
            for (int r = 0; r < R; ++r) acc[t][u][r] = __builtin_fmaf(part[r], s, acc[t][u][r]);
          }
        }
      }
    }
  };

  const int whole = K / kFp4Chunk;
  int chunk = wave;
  for (; chunk + (DEPTH - 1) * WAVES < whole; chunk += DEPTH * WAVES) {
    Chunk c[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(c[d], chunk + d * WAVES);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) multiply(c[d], 4);
  }
  for (; chunk < whole; chunk += WAVES) {
    Chunk c;
    load(c, chunk);
    multiply(c, 4);
  }
  // The blocks behind the last whole chunk, by the wave whose turn it is.
  const int rest = K / kFp4Block - whole * 4;
  if (rest > 0 && chunk == whole) {
    Chunk c;
    const int64_t k = static_cast<int64_t>(whole) * kFp4Chunk;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      c.w[t] = uint4_v{0, 0, 0, 0};
      c.s[t] = 0;
      if (g < rest) c.w[t] = *reinterpret_cast<const uint4_v *>(wrow[t] + k / 2 + g * 16);
      for (int i = 0; i < rest; ++i) c.s[t] |= static_cast<uint32_t>(srow[t][whole * 4 + i]) << (8 * i);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c.x[t][i] = i < rest ? *reinterpret_cast<const half8_t *>(xrow[t] + k + i * kFp4Block) : half8_t{};
    multiply(c, rest);
  }

  // One row of x: its sums are in the first register of lanes 0 .. 15.
  constexpr int kLanes = FULL ? 64 : 16;
  constexpr int kSums = NT * MT * R * kLanes;
  __shared__ float part[WAVES][kSums];
  if (lane < kLanes) {
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
      for (int b = 0; b < MT; ++b)
#pragma unroll
        for (int r = 0; r < R; ++r) part[wave][((a * MT + b) * R + r) * kLanes + lane] = acc[a][b][r];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kSums; i += WAVES * 64) {
    float sum = part[0][i];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += part[w][i];
    const int l = i % kLanes, r = i / kLanes % R, b = i / (kLanes * R) % MT, a = i / (kLanes * R * MT);
    const int m = m0 + b * 16 + (l >> 4) * 4 + r, n = n0 + a * 16 + (l & 15);
    if (m < M && n < N) y[static_cast<int64_t>(m) * N + n] = __builtin_bit_cast(uint16_t, round_out<DT>(sum));
  }
}

// ---- quantiser -------------------------------------------------------------
// Two lanes hold a block, 16 numbers each.  The scale is the least power of two
// with amax <= 6 * scale (from 2^-127 on), so no number is beyond the format's
// largest.  K % 32 == 0: blocks, numbers and scales are numbered straight
// through the matrix.  Dividing by the scale is exact, and one conversion
// rounds to the nearest number, ties to even.
constexpr int kQuantThreads = 256;
template <int DT>
__global__ void __launch_bounds__(kQuantThreads)
quantize_fp4_kernel(const uint16_t *__restrict__ x, uint8_t *__restrict__ q, uint8_t *__restrict__ scale, int64_t halves) {
  const int64_t half = static_cast<int64_t>(blockIdx.x) * kQuantThreads + threadIdx.x;
  if (half >= halves) return;  // both lanes of a block alike
  const uint4_v *src = reinterpret_cast<const uint4_v *>(x + half * 16);
  const uint4_v v[2] = {src[0], src[1]};
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    m2 = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2_v, m2),
                                                                __builtin_bit_cast(ushort2_v, v[i / 4][i % 4] & 0x7fff7fffu)));
  uint32_t top = m2 & 0xffffu;
  if ((m2 >> 16) > top) top = m2 >> 16;
  const uint32_t other = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(top), 0xB1, 0xf, 0xf, false));
  if (other > top) top = other;
  // amax = f 2^e: the scale is 2^(e - 2) for f <= 1.5 and 2^(e - 1) above.
  const uint32_t bits = __builtin_bit_cast(uint32_t, widen_in<DT>(static_cast<uint16_t>(top)));
  const bool finite = bits < 0x7f800000u;
  const int up = static_cast<int>((bits + 0x3fffffu) >> 23) - 2;
  const uint32_t s = finite ? static_cast<uint32_t>(up > 0 ? up : 0) : 255u;
  const float inv = __builtin_bit_cast(float, (254u - s) << 23);  // 1 / scale, a normal number for s <= 253
  uint2_v out = {0, 0};
  if (finite) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t w = 0;
      const auto pair = [&](int j, float &a, float &b) {
        a = widen_in<DT>(static_cast<uint16_t>(v[i][j])) * inv;
        b = widen_in<DT>(static_cast<uint16_t>(v[i][j] >> 16)) * inv;
      };
      float a, b;
      pair(0, a, b);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a, b, 1.0f, 0);
      pair(1, a, b);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a, b, 1.0f, 1);
      pair(2, a, b);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a, b, 1.0f, 2);
      pair(3, a, b);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a, b, 1.0f, 3);
      out[i] = w;
    }
  }
  *reinterpret_cast<uint2_v *>(q + half * 8) = out;
  if ((threadIdx.x & 1) == 0) scale[half >> 1] = static_cast<uint8_t>(s);
}

template <int DT, int MT, int NT, int WAVES, int DEPTH, bool FULL>
hipError_t launch_gemv(const void *x, const void *W, const void *sW, void *y, int M, int N, int K, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((N + NT * 16 - 1) / (NT * 16)), static_cast<unsigned>((M + MT * 16 - 1) / (MT * 16)));
  hipLaunchKernelGGL((gemv_fp4_kernel<DT, MT, NT, WAVES, DEPTH, FULL>), grid, dim3(WAVES * 64), 0, stream,
                     static_cast<const uint16_t *>(x), static_cast<const uint8_t *>(W), static_cast<const uint8_t *>(sW),
                     static_cast<uint16_t *>(y), M, N, K);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_gemv_dt(const void *x, const void *W, const void *sW, void *y, int M, int N, int K, hipStream_t stream) {
  if (M == 1) return launch_gemv<DT, 1, 1, 8, 2, false>(x, W, sW, y, M, N, K, stream);
  if (M <= 16) return launch_gemv<DT, 1, 1, 8, 2, true>(x, W, sW, y, M, N, K, stream);
  if (M <= 32) return launch_gemv<DT, 2, 1, 8, 2, true>(x, W, sW, y, M, N, K, stream);
  return launch_gemv<DT, 4, 1, 8, 1, true>(x, W, sW, y, M, N, K, stream);
}

}  // namespace

hipError_t launch_gemv_fp4(int dtype, const void *x, const void *W, const void *sW, void *y, int M, int N, int K,
                           hipStream_t stream) {
  return dtype == kBF16 ? launch_gemv_dt<kBF16>(x, W, sW, y, M, N, K, stream)
                        : launch_gemv_dt<kF16>(x, W, sW, y, M, N, K, stream);
}

hipError_t launch_quantize_fp4(int dtype, const void *x, void *q, void *scale, int64_t elements, hipStream_t stream) {
  const int64_t halves = elements / 16;
  const dim3 grid(static_cast<unsigned>((halves + kQuantThreads - 1) / kQuantThreads));
  const auto kernel = dtype == kBF16 ? quantize_fp4_kernel<kBF16> : quantize_fp4_kernel<kF16>;
  hipLaunchKernelGGL(kernel, grid, dim3(kQuantThreads), 0, stream, static_cast<const uint16_t *>(x),
                     static_cast<uint8_t *>(q), static_cast<uint8_t *>(scale), halves);
  return hipGetLastError();
}

}  // namespace gt
