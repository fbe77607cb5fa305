// stream.hip -- products of few rows with a weight matrix that is read once:
// block-scaled e4m3 weights (one matrix, or one per group), and 16-bit
// weights of several groups.
//
//   D[t, n] = sum_k x[t, k] W[n, k]                                   16-bit
//   D[t, n] = sum_b sx[t, b] sw[n / r, b] sum_{k in b} x[t, k] W[n, k]  8-bit
//
// Bound by reading W: a workgroup owns 16 or 32 rows of W and all of a unit's
// rows of x (up to 16 of them), so each byte of W is read once per unit.  Its
// waves split K in steps of 128 bytes of a row, which for 8-bit operands is
// one scale block: a step is two 16x16x32 MFMAs of 16-bit numbers or four of
// widened 8-bit ones (fp8_common.hpp), W rows first, so that lane l holds
// outputs n = 4 (l / 16) + e of row l % 16 of x.  Its 8-bit sum is scaled by
// sx[row] * sw in FP32 as it joins the wave's running sum.  Lane l loads two
// 16-byte pieces of row l % 16, pieces l / 16 and 4 + l / 16 of the step's
// eight, so that an instruction reads 64 contiguous bytes of each of 16 rows;
// operands go straight to registers, UNROLL steps of each wave in flight.
// Rows past the last and bytes past the row's end read as zeros through the
// buffer descriptor's range.  The waves' sums meet in LDS and are added in
// wave order, so results do not depend on timing.
//
// Groups: unit u of the launch is found from the offsets in device memory
// (groups.hpp); workgroups past the last unit return at once.
#include "fp8_common.hpp"
#include "groups.hpp"
#include "kernels.hpp"

namespace gt {

namespace {

constexpr int kStepBytes = 128;  // bytes of a row per step

struct StreamArgs {
  const uint8_t *x, *w;
  const float *sx, *sw;
  const int *offsets;
  uint16_t *d;
  int T, N, E;
  int row_bytes;  // of x and W
  int blocks_n;   // workgroups along W's rows
};

// IN: kF16, kBF16 (16-bit operands) or kE4m3.  SW: rows of W per scale (128 or
// 1).  PB: 16-row blocks of W per workgroup.
constexpr int kE4m3 = 2;
template <int IN, int OUT, int PB, int WAVES, int UNROLL, bool GROUPED, int SW>
__global__ void __launch_bounds__(WAVES * 64) stream_kernel(StreamArgs a) {
  constexpr bool kScaled = IN == kE4m3;
  constexpr int kRows = 16 * PB;
  __shared__ float partial[WAVES][kStreamUnit][kRows + 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.blocks_n)) * kRows;
  const int unit = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.blocks_n));
  GroupUnit g{0, unit * kStreamUnit, a.T};
  if constexpr (GROUPED) {
    if (!find_unit(a.offsets, a.E, a.T, kStreamUnit, unit, &g)) return;
  }
  const int rows = min(kStreamUnit, g.end - g.row);
  const uint32_t rb = static_cast<uint32_t>(a.row_bytes);
  const int steps = (a.row_bytes + kStepBytes - 1) / kStepBytes;

  // Byte ranges, so that what lies outside reads as zeros.
  auto range = [](const void *p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, static_cast<int>(bytes), 0x00020000);
  };
  auto load16 = [](__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(int4_t, __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(off), 0, 0));
  };
  const int w_rows = min(kRows, a.N - n0);
  const int64_t w_row = static_cast<int64_t>(g.group) * a.N + n0;
  const auto rsrc_w = range(a.w + w_row * a.row_bytes, static_cast<int64_t>(w_rows) * rb);
  const auto rsrc_x = range(a.x + static_cast<int64_t>(g.row) * a.row_bytes, static_cast<int64_t>(rows) * rb);
  const int frow = lane & 15;
  const int fgrp = lane >> 4;
  const uint32_t piece = static_cast<uint32_t>(fgrp) * 16;
  const uint32_t lane_off = static_cast<uint32_t>(frow) * rb + piece;

  // Scales of this lane's rows of x, and of the rows of W of its outputs: 4
  // steps' at a time, from one 16-byte load (4-byte aligned is enough).
  __amdgpu_buffer_rsrc_t rsrc_sx, rsrc_sw;
  if constexpr (kScaled) {
    rsrc_sx = range(a.sx + static_cast<int64_t>(g.row) * steps, static_cast<int64_t>(rows) * steps * 4);
    const int64_t sw_row = SW == 1 ? w_row
                                   : static_cast<int64_t>(g.group) * ((a.N + kScaleBlock - 1) / kScaleBlock) + n0 / kScaleBlock;
    rsrc_sw = range(a.sw + sw_row * steps, static_cast<int64_t>(SW == 1 ? w_rows : 1) * steps * 4);
  }
  static_assert(UNROLL <= 4, "the scales of one 16-byte load");

  float4_t acc[PB];
#pragma unroll
  for (int p = 0; p < PB; ++p) acc[p] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  // Workgroups that run side by side on an XCD (every eighth) start their
  // waves at different places of K, so that they do not all ask for the same
  // lines of x at once.
  const int first = static_cast<int>((static_cast<unsigned>(wave) + (blockIdx.x >> 3)) % WAVES);
  for (int s0 = first * UNROLL; s0 < steps; s0 += WAVES * UNROLL) {
    int4_t wv[UNROLL][PB][2], xv[UNROLL][2];
    float4_t sxv{}, swv[SW == 1 ? 4 * PB : 1];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = static_cast<uint32_t>(s0 + u) * kStepBytes + 64u * h;
        const uint32_t off = at + piece < rb ? lane_off + at : kOobOffset;
#pragma unroll
        for (int p = 0; p < PB; ++p) wv[u][p][h] = load16(rsrc_w, off + 16u * p * rb);
        xv[u][h] = load16(rsrc_x, off);
      }
    }
    if constexpr (kScaled) {
      sxv = __builtin_bit_cast(float4_t, load16(rsrc_sx, static_cast<uint32_t>(frow * steps + s0) * 4u));
#pragma unroll
      for (int r = 0; r < (SW == 1 ? 4 * PB : 1); ++r) {
        const int row = SW == 1 ? 16 * (r / 4) + 4 * fgrp + r % 4 : 0;
        swv[r] = __builtin_bit_cast(float4_t, load16(rsrc_sw, static_cast<uint32_t>(row * steps + s0) * 4u));
      }
    }
    // Every load of the steps is issued before the first is waited for.
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      // A step past the end multiplies zeros; its scales, which belong to the
      // next row, may be anything and count as zero.
      const bool past = s0 + u >= steps;
      WideOperand wide_x;
      if constexpr (kScaled) wide_x = widen_fp8(join(xv[u][0], xv[u][1]));
#pragma unroll
      for (int p = 0; p < PB; ++p) {
        if constexpr (kScaled) {
          // 16 rows of W in one chain 1x4096x14336 10.9 us, 4x28672x4096 24.3; 32
          // rows in two 256 rows in 64 groups x 2048 x 4096 99.4.
          const float4_t v = mfma_wide<PB == 1 ? 2 : 1>(widen_fp8(join(wv[u][p][0], wv[u][p][1])), wide_x);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float scale = sxv[u] * swv[SW == 1 ? 4 * p + e : 0][u];
            acc[p][e] = __builtin_fmaf(v[e], past ? 0.0f : scale, acc[p][e]);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (IN == kF16)
              acc[p] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, wv[u][p][h]),
                                                              __builtin_bit_cast(half8_t, xv[u][h]), acc[p], 0, 0, 0);
            else
              acc[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wv[u][p][h]),
                                                               __builtin_bit_cast(bf16x8_t, xv[u][h]), acc[p], 0, 0, 0);
          }
        }
      }
    }
  }

#pragma unroll
  for (int p = 0; p < PB; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e) partial[wave][frow][16 * p + 4 * fgrp + e] = acc[p][e];
  __syncthreads();
  for (int i = threadIdx.x; i < kStreamUnit * kRows; i += WAVES * 64) {
    const int t = i / kRows, n = i % kRows;
    if (t >= rows || n >= w_rows) continue;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += partial[w][t][n];
    a.d[static_cast<int64_t>(g.row + t) * a.N + n0 + n] = __builtin_bit_cast(uint16_t, round_out<OUT>(sum));
  }
}

template <int IN, int OUT, int PB, int WAVES, int UNROLL, bool GROUPED, int SW>
hipError_t launch_one(StreamArgs a, int64_t units, hipStream_t stream) {
  a.blocks_n = (a.N + 16 * PB - 1) / (16 * PB);
  const dim3 grid(static_cast<unsigned>(units * a.blocks_n));
  hipLaunchKernelGGL((stream_kernel<IN, OUT, PB, WAVES, UNROLL, GROUPED, SW>), grid, dim3(WAVES * 64), 0, stream, a);
  return hipGetLastError();
}

// The launch shape.  Measured (MI355X; PB x WAVES x UNROLL):
//  * Many groups make many workgroups of little work: small ones of 32 rows of
//    W with few loads in flight each, so that more of them share a CU (8 bits,
//    a row in each of 64 groups x 2048 x 4096: 1x8x4 109 us, 2x8x4 115, 2x4x2 93;
//    16-bit 32 rows x 2048 x 2048 40.9, 41.8 and 38.7).
//  * Else 16 rows of W, and 2 steps in flight instead of 4 where that leaves
//    the slowest wave fewer steps (1x4096x14336, 112 steps: 11.8 -> 10.9 us).
int stream_blocks(int64_t units, int64_t N, int num_cus) {
  return units * ((N + 31) / 32) >= 2 * static_cast<int64_t>(num_cus) ? 2 : 1;
}

template <int IN, int OUT, bool GROUPED, int SW>
hipError_t launch_rows(const StreamArgs &a, int64_t units, int num_cus, hipStream_t stream) {
  if constexpr (GROUPED) {
    if (stream_blocks(units, a.N, num_cus) == 2) return launch_one<IN, OUT, 2, 4, 2, GROUPED, SW>(a, units, stream);
  }
  const int steps = (a.row_bytes + kStepBytes - 1) / kStepBytes;
  const bool two = (steps + 15) / 16 * 2 < (steps + 31) / 32 * 4;
  return two ? launch_one<IN, OUT, 1, 8, 2, GROUPED, SW>(a, units, stream)
             : launch_one<IN, OUT, 1, 8, 4, GROUPED, SW>(a, units, stream);
}

}  // namespace

int grouped_stream_blocks(int64_t T, int64_t N, int64_t E, int num_cus) {
  return stream_blocks(unit_bound(T, E, kStreamUnit), N, num_cus);
}

hipError_t launch_stream_fp8(int out, const void *x, const float *sx, const void *w, const float *sw, int w_scale_rows,
                             void *d, int M, int N, int K, hipStream_t stream) {
  const StreamArgs a{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(w), sx, sw, nullptr,
                     static_cast<uint16_t *>(d), M, N, 1, K, 0};
  static_assert(kStreamRows <= kStreamUnit, "one unit");
  if (w_scale_rows == 1)
    return out == kBF16 ? launch_rows<kE4m3, kBF16, false, 1>(a, 1, 0, stream)
                        : launch_rows<kE4m3, kF16, false, 1>(a, 1, 0, stream);
  return out == kBF16 ? launch_rows<kE4m3, kBF16, false, kScaleBlock>(a, 1, 0, stream)
                      : launch_rows<kE4m3, kF16, false, kScaleBlock>(a, 1, 0, stream);
}

hipError_t launch_stream_grouped(int dtype, const void *x, const void *w, const int *offsets, void *d, int T, int N,
                                 int K, int E, int num_cus, hipStream_t stream) {
  const StreamArgs a{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(w), nullptr, nullptr, offsets,
                     static_cast<uint16_t *>(d), T, N, E, 2 * K, 0};
  const int64_t units = unit_bound(T, E, kStreamUnit);
  return dtype == kBF16 ? launch_rows<kBF16, kBF16, true, kScaleBlock>(a, units, num_cus, stream)
                        : launch_rows<kF16, kF16, true, kScaleBlock>(a, units, num_cus, stream);
}

hipError_t launch_stream_grouped_fp8(int out, const void *x, const float *sx, const void *w, const float *sw,
                                     const int *offsets, void *d, int T, int N, int K, int E, int num_cus,
                                     hipStream_t stream) {
  const StreamArgs a{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(w), sx, sw, offsets,
                     static_cast<uint16_t *>(d), T, N, E, K, 0};
  const int64_t units = unit_bound(T, E, kStreamUnit);
  return out == kBF16 ? launch_rows<kE4m3, kBF16, true, kScaleBlock>(a, units, num_cus, stream)
                      : launch_rows<kE4m3, kF16, true, kScaleBlock>(a, units, num_cus, stream);
}

}  // namespace gt
