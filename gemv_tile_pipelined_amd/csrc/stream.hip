// stream.hip -- products of few rows with a weight matrix that is read once:
// block-scaled e4m3 weights (one matrix, or one per group), and 16-bit
// weights of several groups.
//
//   D[t, n] = sum_k x[t, k] W[n, k]                                   16-bit
//   D[t, n] = sum_b sx[t, b] sw[n / r, b] sum_{k in b} x[t, k] W[n, k]  8-bit
//
// Bound by reading W: a workgroup owns 16 rows of W and all of a unit's rows
// of x (up to 16 QB of them), so each byte of W is read once per unit.  Its
// waves split K in steps of 128 bytes of a row, which for 8-bit operands is
// one scale block: a step is one 16x16x128 MFMA per 16 rows of x (two
// 16x16x32 of 16-bit numbers), W rows first, so that lane l holds outputs
// n = 4 (l / 16) + e of row l % 16 of x.  Its 8-bit sum is scaled by
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
constexpr int kStreamRows = 16;  // rows of W per workgroup
constexpr int kUnroll = 4;

struct StreamArgs {
  const uint8_t *x, *w;
  const float *sx, *sw;
  const int *offsets;
  uint16_t *d;
  int T, N, E;
  int row_bytes;  // of x and W
  int blocks_n;   // 16-row blocks of W
};

// IN: kF16, kBF16 (16-bit operands) or kE4m3.  SW: rows of W per scale (128 or 1).
constexpr int kE4m3 = 2;
template <int IN, int OUT, int QB, int WAVES, bool GROUPED, int SW>
__global__ void __launch_bounds__(WAVES * 64) stream_kernel(StreamArgs a) {
  constexpr bool kScaled = IN == kE4m3;
  __shared__ float partial[WAVES][16 * QB][kStreamRows + 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.blocks_n)) * kStreamRows;
  const int unit = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.blocks_n));
  GroupUnit g{0, unit * 16 * QB, a.T};
  if constexpr (GROUPED) {
    if (!find_unit(a.offsets, a.E, a.T, 16 * QB, unit, &g)) return;
  }
  const int rows = min(16 * QB, g.end - g.row);
  const uint32_t rb = static_cast<uint32_t>(a.row_bytes);
  const int steps = (a.row_bytes + kStepBytes - 1) / kStepBytes;

  const int64_t w_row = static_cast<int64_t>(g.group) * a.N + n0;
  const auto rsrc_w = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(a.w + w_row * a.row_bytes), 0, static_cast<int>(min(kStreamRows, a.N - n0) * rb), 0x00020000);
  const auto rsrc_x = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(a.x + static_cast<int64_t>(g.row) * a.row_bytes), 0, static_cast<int>(rows * rb), 0x00020000);
  const int frow = lane & 15;
  const uint32_t piece = static_cast<uint32_t>(lane >> 4) * 16;
  const uint32_t lane_off = static_cast<uint32_t>(frow) * rb + piece;

  // Scales of this lane's rows: rows past the last repeat the last one's (their
  // sums are zeros, or are not stored).
  const float *sx[QB];
  const float *sw[4];
  if constexpr (kScaled) {
#pragma unroll
    for (int q = 0; q < QB; ++q) sx[q] = a.sx + static_cast<int64_t>(g.row + min(16 * q + frow, rows - 1)) * steps;
    if constexpr (SW == 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sw[e] = a.sw + static_cast<int64_t>(min(n0 + 4 * (lane >> 4) + e, a.N - 1)) * steps;
    } else {
      sw[0] = a.sw + (static_cast<int64_t>(g.group) * ((a.N + kScaleBlock - 1) / kScaleBlock) + n0 / kScaleBlock) * steps;
    }
  }

  float4_t acc[QB];
#pragma unroll
  for (int q = 0; q < QB; ++q) acc[q] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = wave * kUnroll; s0 < steps; s0 += WAVES * kUnroll) {
    int4_t wv[kUnroll][2], xv[kUnroll][QB][2];
    float sxv[kUnroll][QB], swv[kUnroll][SW == 1 ? 4 : 1];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = static_cast<uint32_t>(s0 + u) * kStepBytes + 64u * h;
        const uint32_t off = at + piece < rb ? lane_off + at : kOobOffset;
        wv[u][h] = __builtin_bit_cast(int4_t, __builtin_amdgcn_raw_buffer_load_b128(rsrc_w, off, 0, 0));
#pragma unroll
        for (int q = 0; q < QB; ++q)
          xv[u][q][h] = __builtin_bit_cast(int4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                       rsrc_x, at + piece < rb ? off + 16u * q * rb : kOobOffset, 0, 0));
      }
      if constexpr (kScaled) {
        const int b = min(s0 + u, steps - 1);
#pragma unroll
        for (int q = 0; q < QB; ++q) sxv[u][q] = sx[q][b];
#pragma unroll
        for (int e = 0; e < (SW == 1 ? 4 : 1); ++e) swv[u][e] = sw[e][b];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (s0 + u >= steps) break;  // uniform; a step past the end would add zeros
#pragma unroll
      for (int q = 0; q < QB; ++q) {
        if constexpr (kScaled) {
          const float4_t p =
              mfma_fp8(join(wv[u][0], wv[u][1]), join(xv[u][q][0], xv[u][q][1]), float4_t{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[q][e] = __builtin_fmaf(p[e], sxv[u][q] * swv[u][SW == 1 ? e : 0], acc[q][e]);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (IN == kF16)
              acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, wv[u][h]),
                                                              __builtin_bit_cast(half8_t, xv[u][q][h]), acc[q], 0, 0, 0);
            else
              acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wv[u][h]),
                                                               __builtin_bit_cast(bf16x8_t, xv[u][q][h]), acc[q], 0, 0, 0);
          }
        }
      }
    }
  }

#pragma unroll
  for (int q = 0; q < QB; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) partial[wave][16 * q + frow][4 * (lane >> 4) + e] = acc[q][e];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * QB * kStreamRows; i += WAVES * 64) {
    const int t = i / kStreamRows, n = i % kStreamRows;
    if (t >= rows || n0 + n >= a.N) continue;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += partial[w][t][n];
    a.d[static_cast<int64_t>(g.row + t) * a.N + n0 + n] = __builtin_bit_cast(uint16_t, round_out<OUT>(sum));
  }
}

template <int IN, int OUT, int QB, int WAVES, bool GROUPED, int SW>
hipError_t launch_one(const StreamArgs &a, int64_t units, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(units * a.blocks_n));
  hipLaunchKernelGGL((stream_kernel<IN, OUT, QB, WAVES, GROUPED, SW>), grid, dim3(WAVES * 64), 0, stream, a);
  return hipGetLastError();
}

// 4 steps or more for a wave, as far as 4 to 16 waves allow; 16 waves of 64
// rows would not leave two workgroups their LDS.
template <int IN, int OUT, int QB, bool GROUPED, int SW>
hipError_t launch_waves(const StreamArgs &a, int64_t units, hipStream_t stream) {
  const int steps = (a.row_bytes + kStepBytes - 1) / kStepBytes;
  if (steps >= 16 * kUnroll && QB < 4) return launch_one<IN, OUT, QB, 16, GROUPED, SW>(a, units, stream);
  if (steps >= 8 * kUnroll) return launch_one<IN, OUT, QB, 8, GROUPED, SW>(a, units, stream);
  return launch_one<IN, OUT, QB, 4, GROUPED, SW>(a, units, stream);
}

template <int IN, int OUT, bool GROUPED, int SW>
hipError_t launch_rows(const StreamArgs &a, int rows, int64_t units, hipStream_t stream) {
  if (rows <= 16) return launch_waves<IN, OUT, 1, GROUPED, SW>(a, units, stream);
  if (rows <= 32) return launch_waves<IN, OUT, 2, GROUPED, SW>(a, units, stream);
  return launch_waves<IN, OUT, 4, GROUPED, SW>(a, units, stream);
}

}  // namespace

hipError_t launch_stream_fp8(int out, const void *x, const float *sx, const void *w, const float *sw, int w_scale_rows,
                             void *d, int M, int N, int K, hipStream_t stream) {
  const StreamArgs a{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(w), sx, sw, nullptr,
                     static_cast<uint16_t *>(d), M, N, 1, K, (N + kStreamRows - 1) / kStreamRows};
  const int rows = M <= 16 ? 16 : M <= 32 ? 32 : 64;
  const int64_t units = (M + rows - 1) / rows;
  if (w_scale_rows == 1)
    return out == kBF16 ? launch_rows<kE4m3, kBF16, false, 1>(a, rows, units, stream)
                        : launch_rows<kE4m3, kF16, false, 1>(a, rows, units, stream);
  return out == kBF16 ? launch_rows<kE4m3, kBF16, false, kScaleBlock>(a, rows, units, stream)
                      : launch_rows<kE4m3, kF16, false, kScaleBlock>(a, rows, units, stream);
}

hipError_t launch_stream_grouped(int dtype, const void *x, const void *w, const int *offsets, void *d, int T, int N,
                                 int K, int E, int rows, hipStream_t stream) {
  const StreamArgs a{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(w), nullptr, nullptr, offsets,
                     static_cast<uint16_t *>(d), T, N, E, 2 * K, (N + kStreamRows - 1) / kStreamRows};
  const int64_t units = unit_bound(T, E, rows);
  return dtype == kBF16 ? launch_rows<kBF16, kBF16, true, kScaleBlock>(a, rows, units, stream)
                        : launch_rows<kF16, kF16, true, kScaleBlock>(a, rows, units, stream);
}

hipError_t launch_stream_grouped_fp8(int out, const void *x, const float *sx, const void *w, const float *sw,
                                     const int *offsets, void *d, int T, int N, int K, int E, int rows,
                                     hipStream_t stream) {
  const StreamArgs a{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(w), sx, sw, offsets,
                     static_cast<uint16_t *>(d), T, N, E, K, (N + kStreamRows - 1) / kStreamRows};
  const int64_t units = unit_bound(T, E, rows);
  return out == kBF16 ? launch_rows<kE4m3, kBF16, true, kScaleBlock>(a, rows, units, stream)
                      : launch_rows<kE4m3, kF16, true, kScaleBlock>(a, rows, units, stream);
}

}  // namespace gt
