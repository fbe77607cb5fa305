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
// The product reads 17 bytes of W for 32 numbers and is bound by that for one token: each
// is read once by up to 48 rows of x, by fewer where gemv_shape has several workgroups
// read the same.  One v_cvt_scalef32_pk_*_fp4 turns a byte into two numbers of x's format
// times the scale, and 16-bit MFMAs (16x16x32) multiply exactly and add in FP32.
// Lane n + 16 g of a wave holds the whole block g of four that follow one another
// in row n, and as many of x: an MFMA takes 8 numbers of each of the four blocks.
//
// That is exact where scaled numbers are numbers of the 16-bit format: scales of
// 2^-125 to 2^125 in bf16, 2^-23 to 2^13 in half precision, which weights have.
// Four blocks with another scale among them in a workgroup's rows (blocks of zeros have
// the smallest), and those at a ragged end of K, take the exact way for any scale: numbers
// converted without it, one MFMA for each block, whose sum is then scaled in FP32.
// That wants all four lane rows to hold 8 numbers each of one block, which is the
// transpose of 4 x 4 dwords across lane rows (two v_permlane32_swap and two
// v_permlane16_swap), of W and of x.  It costs up to half as much again (1, 27 and 64 rows
// of 4096x14336, 8195x4128 and 4096x14336: 8.0, 10.9 and 18.0 us without a block of zeros,
// 8.8, 12.2 and 20.6 with one in 1000, 10.7, 14.1 and 25.9 with one in 100, 11.7, 14.4 and
// 27.9 with zeros only), and sums come in another order.
//
// Loads go straight to LDS.  A wave's 64 x 16 bytes are 16 rows of 64 bytes: where
// neighbouring lanes load from the rows of an MFMA's operand, 16 different cache
// lines each, a CU gets 10 bytes a cycle (1x4096x14336 11.3 us however deep the
// prefetch); with neighbouring lanes along the rows it is what memory gives.  LDS
// hands them to the lanes that multiply.  1x4096x14336 then takes 7.3 us of which 5.9
// are its bytes at a large copy's rate; 27x8195x4128 10.4, where x, read by every
// workgroup, is twice W.
#include "device_common.hpp"
#include "kernels.hpp"
#include "wave_ops.hpp"

namespace gt {

namespace {

typedef unsigned short ushort2_v __attribute__((ext_vector_type(2)));

constexpr int kFp4Block = 32;   // numbers that share a scale; also the K of one MFMA
constexpr int kFp4Chunk = 128;  // columns that a wave takes at a time

// The 8 numbers of a dword times a scale (a power of two) in x's format.
template <int DT>
__device__ inline half8_t widen_fp4(uint32_t v, float scale) {
  half8_t w;
  if constexpr (DT == kF16) {
    const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, scale, 0);
    const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, scale, 1);
    const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, scale, 2);
    const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, scale, 3);
    w = half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3);
    w = __builtin_bit_cast(half8_t, bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]});
  }
  return w;
}

// Scale bytes with which every scaled number is one of the 16-bit format.
template <int DT>
__device__ inline bool scale_fits(uint32_t s) {
  constexpr uint32_t kLow = DT == kF16 ? 127 - 23 : 127 - 125, kHigh = DT == kF16 ? 127 + 13 : 127 + 125;
  return s - kLow <= kHigh - kLow;
}

template <int DT>
__device__ inline float4_t mfma_16x16x32(half8_t a, half8_t b, float4_t c) {
  if constexpr (DT == kF16) return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// 4 x 4 dwords across the four lane rows: v[i] of lane row g <-> v[g] of row i.
__device__ inline uint4_v transpose_rows(uint4_v v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return uint4_v{c[0], c[1], d[0], d[1]};
}

// 2^(s - 127): the byte as an FP32 exponent, but for 0 (2^-127, below the normal
// numbers) and 255 (NaN).
__device__ inline float scale_of(uint32_t s) {
  const uint32_t bits = s << 23;
  const float f = __builtin_bit_cast(float, bits > 0x00400000u ? bits : 0x00400000u);
  return s == 0xffu ? __builtin_nanf("") : f;
}

// What lane row i holds, in every lane row, for i = 0 .. 3.
__device__ inline float4_t spread_rows(float v) {
  const int lane = threadIdx.x & 15;
  return float4_t{__shfl(v, lane), __shfl(v, lane + 16), __shfl(v, lane + 32), __shfl(v, lane + 48)};
}

// A workgroup has NT * 16 rows of W and up to XQ * 4 rows of x.  Its waves take
// the chunks of K in turn; each has a ring of its own in LDS, DEPTH chunks of W and
// x on their way, and waits for its own loads only.  Loads outside the matrices
// (rows past the last, the end of a ragged K, chunks past the last) go to an offset
// that buffer loads answer with zeros, so the number in flight is always the same.
// The scales of the workgroup's rows are in LDS too, 16384 columns at a time (8192
// where there are more than 32 rows).  The waves' sums meet in LDS and are added in
// wave order.
//
// Places in LDS, in 16-byte pieces.  W: piece g of row n at 4 n + (g ^ (n >> 2)), so
// that the 16 rows' pieces g are spread over all banks.  x: piece p (of 16) of row m
// at 16 m + (p ^ (m & 15)), likewise.
template <int DT, int XQ, int NT, int WAVES, int DEPTH>
__global__ void __launch_bounds__(WAVES * 64)
gemv_fp4_kernel(const uint16_t *__restrict__ x, const uint8_t *__restrict__ W, const uint8_t *__restrict__ sW,
                uint16_t *__restrict__ y, int M, int N, int K) {
  constexpr int MT = (XQ + 3) / 4;               // blocks of 16 rows of x
  constexpr int kChains = NT * MT == 1 ? 2 : 1;  // of MFMAs that wait for one another
  constexpr int kSums = NT * MT * 256;
  constexpr int kLoads = NT + XQ;  // of a chunk, 1 KiB each
  constexpr int kSegment = NT <= 2 ? 128 : 64;    // chunks whose scales are in LDS
  constexpr int kScaleRow = kSegment * 4 + 16;  // bytes for a row's scales and their place within 16
  static_assert(kSums * 4 <= DEPTH * kLoads * 1024, "the sums fit where the ring was");
  __shared__ __attribute__((aligned(16))) char ring[WAVES * DEPTH * kLoads * 1024];
  __shared__ __attribute__((aligned(16))) uint8_t scales[NT * 16 * kScaleRow];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int n0 = static_cast<int>(blockIdx.x) * (NT * 16);
  const int m0 = static_cast<int>(blockIdx.y) * (XQ * 4);
  const int rows = N - n0 < NT * 16 ? N - n0 : NT * 16;
  const int xrows = M - m0 < XQ * 4 ? M - m0 : XQ * 4;
  // Below 2^31 bytes by the limits of the entry point.
  const int4_t wbuf = make_buffer_rsrc(W + static_cast<int64_t>(n0) * (K / 2), static_cast<uint32_t>(rows) * (K / 2));
  const int4_t xbuf = make_buffer_rsrc(x + static_cast<int64_t>(m0) * K, static_cast<uint32_t>(xrows) * K * 2);
  char *const mine = ring + wave * (DEPTH * kLoads * 1024);
  const uint32_t mine_lds = __builtin_amdgcn_readfirstlane(lds_addr(mine));

  // This lane's piece of each load: of W's row lane / 4, and of x's row lane / 16.
  const uint32_t wpiece = (lane & 3) ^ (lane >> 4);
  const uint32_t wat = static_cast<uint32_t>(lane >> 2) * (K / 2) + wpiece * 16;
  const uint32_t wcol = wpiece * kFp4Block;
  auto issue = [&](int chunk, int stage) {
    const int k = chunk * kFp4Chunk;
    const uint32_t to = mine_lds + stage * (kLoads * 1024);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      lds_dma_b128(wbuf, k + wcol < static_cast<uint32_t>(K) ? wat + t * 16 * (K / 2) + k / 2 : kOobOffset, to + t * 1024);
#pragma unroll
    for (int q = 0; q < XQ; ++q) {
      const uint32_t m = q * 4 + g;
      const uint32_t col = k + (i16 ^ (m & 15)) * 8;
      lds_dma_b128(xbuf, col < static_cast<uint32_t>(K) ? (m * K + col) * 2 : kOobOffset, to + (NT + q) * 1024);
    }
  };

  float4_t acc[NT][MT][kChains];
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int b = 0; b < MT; ++b)
#pragma unroll
      for (int r = 0; r < kChains; ++r) acc[a][b][r] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // Where this lane reads: W's piece g of row i16 of a block, x's pieces of row i16
  // (of the last one that has a place where there are fewer: what it gives is not
  // stored).
  const uint32_t wread = (4 * i16 + (g ^ (i16 >> 2))) * 16;
  auto read = [&](const char *stage, uint4_v (&w)[NT], uint4_v (&xv)[MT][4]) {
#pragma unroll
    for (int t = 0; t < NT; ++t) w[t] = *reinterpret_cast<const uint4_v *>(stage + t * 1024 + wread);
#pragma unroll
    for (int u = 0; u < MT; ++u) {
      const int row = u * 16 + i16 < XQ * 4 ? u * 16 + i16 : XQ * 4 - 1;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xv[u][i] = *reinterpret_cast<const uint4_v *>(stage + NT * 1024 + (row * 16 + ((4 * g + i) ^ (row & 15))) * 16);
    }
  };
  auto multiply = [&](const uint4_v (&w)[NT], const uint4_v (&xv)[MT][4], const uint32_t (&s)[NT]) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float scale = __builtin_bit_cast(float, s[t] << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const half8_t b = widen_fp4<DT>(w[t][i], scale);
#pragma unroll
        for (int u = 0; u < MT; ++u)
          acc[t][u][i % kChains] = mfma_16x16x32<DT>(__builtin_bit_cast(half8_t, xv[u][i]), b, acc[t][u][i % kChains]);
      }
    }
  };
  auto multiply_exactly = [&](const uint4_v (&wv)[NT], const uint4_v (&xv)[MT][4], const uint32_t (&sv)[NT]) {
    uint4_v xt[MT][4];
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4_v v = transpose_rows(uint4_v{xv[u][0][j], xv[u][1][j], xv[u][2][j], xv[u][3][j]});
#pragma unroll
        for (int i = 0; i < 4; ++i) xt[u][i][j] = v[i];
      }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint4_v w = transpose_rows(wv[t]);
      const float4_t s = spread_rows(scale_of(sv[t]));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const half8_t b = widen_fp4<DT>(w[i], 1.0f);
#pragma unroll
        for (int u = 0; u < MT; ++u) {
          const float4_t part =
              mfma_16x16x32<DT>(__builtin_bit_cast(half8_t, xt[u][i]), b, float4_t{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[t][u][0][r] = __builtin_fmaf(part[r], s[i], acc[t][u][0][r]);
        }
      }
    }
  };

  const int chunks = (K + kFp4Chunk - 1) / kFp4Chunk, row_blocks = K / kFp4Block;
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) issue(wave + d * WAVES, d);
  int chunk = wave, stage = 0;
  for (int first = 0; first < chunks; first += kSegment) {
    // The scales of the segment.  A row's keep their place within 16 bytes, so that
    // whole pieces are moved wherever it begins.
    const int b0 = first * 4, nb = row_blocks - b0 < kSegment * 4 ? row_blocks - b0 : kSegment * 4;
    const uint8_t *src = sW + static_cast<int64_t>(n0) * row_blocks + b0;
    if (first > 0) __syncthreads();
    const int pieces = (nb + 30) / 16;
    for (int i = threadIdx.x; i < rows * pieces; i += WAVES * 64) {
      const int r = i / pieces, at = (i - r * pieces) * 16;
      const uint8_t *row = src + static_cast<int64_t>(r) * row_blocks;
      const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
      uint8_t *to = scales + r * kScaleRow;
      if (at >= skew && at + 16 <= skew + nb) {
        *reinterpret_cast<uint4_v *>(to + at) = *reinterpret_cast<const uint4_v *>(row + (at - skew));
      } else {
        for (int j = at < skew ? skew : at; j < skew + nb && j < at + 16; ++j) to[j] = row[j - skew];
      }
    }
    __syncthreads();
    const uint8_t *mine_s[NT];  // this lane's rows, by block
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = t * 16 + i16;
      const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(src + static_cast<int64_t>(r) * row_blocks) & 15);
      mine_s[t] = scales + r * kScaleRow + skew - b0;
    }
    const int past = first + kSegment < chunks ? first + kSegment : chunks;
    for (; chunk < past; chunk += WAVES) {
      // Lanes behind the last row or the end of K: zeros of W, any scale but NaN.
      const int block = chunk * 4 + g;
      bool fits = (chunk + 1) * kFp4Chunk <= K;
      uint32_t s[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = t * 16 + i16;
        s[t] = r < rows && block < row_blocks ? mine_s[t][block] : 127u;
        fits &= scale_fits<DT>(s[t]);
      }
      wait_vmcnt<(DEPTH - 1) * kLoads>();
      uint4_v w[NT], xv[MT][4];
      read(mine + stage * (kLoads * 1024), w, xv);
      if (__all(fits)) multiply(w, xv, s);
      else multiply_exactly(w, xv, s);
      wait_lgkmcnt0();  // this stage has been read
      issue(chunk + DEPTH * WAVES, stage);
      stage = stage + 1 == DEPTH ? 0 : stage + 1;
    }
  }
  wait_vmcnt<0>();  // loads past the last chunk, before their places are written
  __syncthreads();
  float(*part)[kSums] = reinterpret_cast<float(*)[kSums]>(ring);
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int b = 0; b < MT; ++b) {
      float4_t sum = acc[a][b][0];
      if constexpr (kChains == 2) sum += acc[a][b][1];
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][((a * MT + b) * 4 + r) * 64 + lane] = sum[r];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < kSums; i += WAVES * 64) {
    const int l = i % 64, r = i / 64 % 4, b = i / 256 % MT, a = i / (256 * MT);
    const int m = m0 + b * 16 + (l >> 4) * 4 + r, n = n0 + a * 16 + (l & 15);
    if (m >= m0 + xrows || n >= N) continue;
    float sum = part[0][i];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += part[w][i];
    y[static_cast<int64_t>(m) * N + n] = __builtin_bit_cast(uint16_t, round_out<DT>(sum));
  }
}

// ---- quantiser -------------------------------------------------------------
// Two lanes hold a block, 16 numbers each.  The scale is the least power of two
// with amax <= 6 * scale (from 2^-127 on), so no number is beyond the format's
// largest.  K % 32 == 0: blocks, numbers and scales are numbered straight
// through the matrix.  Dividing by the scale is exact, and one conversion
// rounds to the nearest number, ties to even.  Bound by memory: 4095 x 14336 in 26.7
// us (5.6 TB/s; some of it is in the last cache already).
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

template <int DT, int XQ, int NT, int WAVES, int DEPTH>
hipError_t launch_gemv(const void *x, const void *W, const void *sW, void *y, int M, int N, int K, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((N + NT * 16 - 1) / (NT * 16)), static_cast<unsigned>((M + XQ * 4 - 1) / (XQ * 4)));
  hipLaunchKernelGGL((gemv_fp4_kernel<DT, XQ, NT, WAVES, DEPTH>), grid, dim3(WAVES * 64), 0, stream,
                     static_cast<const uint16_t *>(x), static_cast<const uint8_t *>(W), static_cast<const uint8_t *>(sW),
                     static_cast<uint16_t *>(y), M, N, K);
  return hipGetLastError();
}

// Rows of x (4 XQ) and of W (16 NT) for a workgroup.  A CU gets 25 bytes a cycle from
// its L2, and a workgroup needs 2 bytes of each of its rows of x and 1/2 of each of W
// for a column, whose unpacking takes about as long again: of the pairs, the one with
// the least rounds * (2 rows of x + 16 NT), of equal ones that with more rows of x.
// Fewer rows of x than there are make several workgroups read the same W, from L2 or
// beyond.  us with what is chosen / with all rows of x and the W of one round:
//   27 rows of x  1024x4096 4.4 / 6.0, 4096x14336 16.5 / 21.6, 8195x4128 10.6 / 10.6, 8192x8192 15.3 / 15.3
//   64            1024x4096 5.1 / 9.5, 4096x14336 22.9 / 34.7, 8195x4128 20.4 / 21.2, 8192x8192 20.3 / 26.7
// Eight waves and the depth that the LDS holds are ahead of fewer waves and more depth.
struct GemvShape {
  int xq, nt;
};
GemvShape gemv_shape(int64_t M, int64_t tiles, int64_t cus) {
  GemvShape best = {2, 1};
  int64_t least = INT64_MAX;
  for (const int xq : {2, 4, 6, 8, 12}) {
    for (int nt = xq == 12 ? 2 : 1; nt <= (xq == 2 ? 2 : 4); ++nt) {
      const int64_t groups = (tiles + nt - 1) / nt * ((M + 4 * xq - 1) / (4 * xq));
      const int64_t cost = (groups + cus - 1) / cus * (2 * (M < 4 * xq ? M : 4 * xq) + 16 * nt);
      if (cost < least || (cost == least && xq > best.xq)) {
        least = cost;
        best = {xq, nt};
      }
    }
    if (4 * xq >= M) break;
  }
  return best;
}

template <int DT>
hipError_t launch_gemv_dt(const void *x, const void *W, const void *sW, void *y, int M, int N, int K, int cus,
                          hipStream_t stream) {
  const int tiles = (N + 15) / 16;
  if (M <= 8) {
    // Several workgroups of few rows of x share a CU: no more than 3 blocks of W, and 2
    // where that does not make one round (1 row: 8195x4128 7.7 us with 1, 7.5 with 2, 6.9
    // with 3; 14336x4096 10.2, 8.3, - and 9.7 with 4; 28672x4096 17.8, 14.8, 15.9, 17.3).
    const int round = (tiles + cus - 1) / cus;
    const int nt = round <= 3 ? round : 2;
    if (M <= 4) {
      // A third stage where a wave has more than four chunks (4096x14336 9.5 us with two,
      // 8.3 with three; 4096x4096 4.2 and 4.5).
      if (nt == 1 && K > 4 * 8 * kFp4Chunk) return launch_gemv<DT, 1, 1, 8, 3>(x, W, sW, y, M, N, K, stream);
      if (nt == 1) return launch_gemv<DT, 1, 1, 8, 2>(x, W, sW, y, M, N, K, stream);
      if (nt == 2) return launch_gemv<DT, 1, 2, 8, 2>(x, W, sW, y, M, N, K, stream);
      return launch_gemv<DT, 1, 3, 8, 2>(x, W, sW, y, M, N, K, stream);
    }
    if (nt == 1) return launch_gemv<DT, 2, 1, 8, 2>(x, W, sW, y, M, N, K, stream);
    // One stage lets three workgroups share a CU (6 rows: 14336x4096 11.1 us with two, 9.0
    // with one; 8192x8192, one round, 10.8 and 11.9).
    if (nt == 2 && round > 2) return launch_gemv<DT, 2, 2, 8, 1>(x, W, sW, y, M, N, K, stream);
    if (nt == 2) return launch_gemv<DT, 2, 2, 8, 2>(x, W, sW, y, M, N, K, stream);
    return launch_gemv<DT, 2, 3, 8, 1>(x, W, sW, y, M, N, K, stream);
  }
  const GemvShape s = gemv_shape(M, tiles, cus);
  switch (s.xq * 8 + s.nt) {
    case 2 * 8 + 1: return launch_gemv<DT, 2, 1, 8, 2>(x, W, sW, y, M, N, K, stream);
    case 2 * 8 + 2: return launch_gemv<DT, 2, 2, 8, 2>(x, W, sW, y, M, N, K, stream);
    case 4 * 8 + 1: return launch_gemv<DT, 4, 1, 8, 2>(x, W, sW, y, M, N, K, stream);
    case 4 * 8 + 2: return launch_gemv<DT, 4, 2, 8, 2>(x, W, sW, y, M, N, K, stream);
    case 4 * 8 + 3: return launch_gemv<DT, 4, 3, 8, 1>(x, W, sW, y, M, N, K, stream);
    case 4 * 8 + 4: return launch_gemv<DT, 4, 4, 8, 1>(x, W, sW, y, M, N, K, stream);
    case 6 * 8 + 1: return launch_gemv<DT, 6, 1, 8, 2>(x, W, sW, y, M, N, K, stream);
    case 6 * 8 + 2: return launch_gemv<DT, 6, 2, 8, 1>(x, W, sW, y, M, N, K, stream);
    case 6 * 8 + 3: return launch_gemv<DT, 6, 3, 8, 1>(x, W, sW, y, M, N, K, stream);
    case 6 * 8 + 4: return launch_gemv<DT, 6, 4, 8, 1>(x, W, sW, y, M, N, K, stream);
    case 8 * 8 + 1: return launch_gemv<DT, 8, 1, 8, 1>(x, W, sW, y, M, N, K, stream);
    case 8 * 8 + 2: return launch_gemv<DT, 8, 2, 8, 1>(x, W, sW, y, M, N, K, stream);
    case 8 * 8 + 3: return launch_gemv<DT, 8, 3, 8, 1>(x, W, sW, y, M, N, K, stream);
    case 8 * 8 + 4: return launch_gemv<DT, 8, 4, 8, 1>(x, W, sW, y, M, N, K, stream);
    case 12 * 8 + 2: return launch_gemv<DT, 12, 2, 8, 1>(x, W, sW, y, M, N, K, stream);
    case 12 * 8 + 3: return launch_gemv<DT, 12, 3, 8, 1>(x, W, sW, y, M, N, K, stream);
    default: return launch_gemv<DT, 12, 4, 4, 1>(x, W, sW, y, M, N, K, stream);
  }
}

}  // namespace

hipError_t launch_gemv_fp4(int dtype, const void *x, const void *W, const void *sW, void *y, int M, int N, int K, int num_cus,
                           hipStream_t stream) {
  return dtype == kBF16 ? launch_gemv_dt<kBF16>(x, W, sW, y, M, N, K, num_cus, stream)
                        : launch_gemv_dt<kF16>(x, W, sW, y, M, N, K, num_cus, stream);
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
