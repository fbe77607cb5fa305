// rows.hip -- tokens' rows to the rows that a router gave them, and back.
//
//   gather        Xs[pos[t,j]] = X[t]
//   combine       Y[t] = sum_j w[t,j] D[pos[t,j]]           (w NULL: ones, the gradient of gather)
//   combine_grad  dD[pos[t,j]] = w[t,j] dY[t],  dw[t,j] = sum_c dY[t,c] D[pos[t,j],c]
//
// Slots whose pos is outside 0 .. rows - 1 are left out.  All three walk over the
// tokens, so a token's own row is read or written once however many experts it
// has, and pos is all that they need.  Sums are in FP32, in the order of j.  Bound
// by memory: 4100 x 8 rows of 4096 bytes are gathered in 30 us (4.9 TB/s), the
// gradient of a combine of 4096 x 8 rows of 2048 takes 58 us (4.9 TB/s; a large copy
// reaches 5.3); 27 x 8 rows are combined in 3.8 us, a launch and its latency.
#include "device_common.hpp"
#include "kernels.hpp"
#include "wave_ops.hpp"

namespace gt {

namespace {

constexpr int kRowThreads = 256;

// Threads of a token: a power of two of at most a workgroup's, one for each 16
// bytes of its row if there are so many; wider rows take several workgroups.
int token_threads_log2(int64_t vecs) {
  int n = 0;
  while (n < 8 && (int64_t{1} << n) < vecs) ++n;
  return n;
}

struct RowPlace {
  int64_t t;
  int v;
};
__device__ inline RowPlace row_place(int log2_threads) {
  const int tokens = kRowThreads >> log2_threads;
  return {static_cast<int64_t>(blockIdx.x) * tokens + (threadIdx.x >> log2_threads),
          (static_cast<int>(blockIdx.y) << log2_threads) + (static_cast<int>(threadIdx.x) & ((1 << log2_threads) - 1))};
}

// Rows of `vecs` 16-byte pieces, and if `scales` of `per_row` FP32 numbers.
__global__ void __launch_bounds__(kRowThreads)
gather_kernel(const uint4_v *__restrict__ X, const float *__restrict__ scale, const int *__restrict__ pos,
              uint4_v *__restrict__ Xs, float *__restrict__ scales, int64_t T, int64_t rows, int vecs, int per_row, int k,
              int log2_threads) {
  const RowPlace p = row_place(log2_threads);
  if (p.t >= T) return;
  const int *at = pos + p.t * k;
  const bool in = p.v < vecs, has_scale = scales != nullptr && p.v < per_row;
  uint4_v x = {0, 0, 0, 0};
  float s = 0.0f;
  if (in) x = X[p.t * vecs + p.v];
  if (has_scale) s = scale[p.t * per_row + p.v];
  for (int j = 0; j < k; ++j) {
    const int r = at[j];
    if (r < 0 || r >= rows) continue;
    if (in) Xs[static_cast<int64_t>(r) * vecs + p.v] = x;
    if (has_scale) scales[static_cast<int64_t>(r) * per_row + p.v] = s;
  }
}

// Four rows at a time, so that their loads are in flight together.
template <int DT>
__global__ void __launch_bounds__(kRowThreads)
combine_kernel(const uint4_v *__restrict__ D, const int *__restrict__ pos, const float *__restrict__ w,
               uint4_v *__restrict__ Y, int64_t T, int64_t rows, int vecs, int k, int log2_threads) {
  const RowPlace p = row_place(log2_threads);
  if (p.t >= T || p.v >= vecs) return;
  const int *at = pos + p.t * k;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
  for (int j0 = 0; j0 < k; j0 += 4) {
    uint4_v d[4];
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d[j] = uint4_v{0, 0, 0, 0};
      f[j] = 0.0f;
      if (j0 + j < k) {
        const int r = at[j0 + j];
        if (r >= 0 && r < rows) {
          d[j] = D[static_cast<int64_t>(r) * vecs + p.v];
          f[j] = w != nullptr ? w[p.t * k + j0 + j] : 1.0f;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a[8];
      widen8<DT>(d[j], a);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(f[j], a[i], sum[i]);
    }
  }
  Y[p.t * vecs + p.v] = round8<DT>(sum);
}

// A token has LANES threads, a workgroup's or a part of a wave; four of its rows at a
// time.
template <int DT, int LANES>
__global__ void __launch_bounds__(kRowThreads)
combine_grad_kernel(const uint4_v *__restrict__ dY, const uint4_v *__restrict__ D, const int *__restrict__ pos,
                    const float *__restrict__ w, uint4_v *__restrict__ dD, float *__restrict__ dw, int64_t T, int64_t rows,
                    int vecs, int k) {
  __shared__ float sums[2][kRowThreads / 64][4];
  const int sub = threadIdx.x % LANES;
  int64_t t = blockIdx.x;
  if constexpr (LANES < kRowThreads) t = t * (kRowThreads / LANES) + threadIdx.x / LANES;
  const bool there = t < T;
  const int *at = pos + t * k;
  int turn = 0;
  for (int j0 = 0; j0 < k; j0 += 4, turn ^= 1) {
    int r[4];
    float f[4], dot[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r[j] = there && j0 + j < k ? at[j0 + j] : -1;
      if (r[j] >= rows) r[j] = -1;
      f[j] = r[j] >= 0 ? w[t * k + j0 + j] : 0.0f;
      dot[j] = 0.0f;
    }
    for (int v = sub; there && v < vecs; v += LANES) {
      float g[8];
      widen8<DT>(dY[t * vecs + v], g);
      uint4_v d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = r[j] >= 0 ? D[static_cast<int64_t>(r[j]) * vecs + v] : uint4_v{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (r[j] < 0) continue;
        float a[8], o[8];
        widen8<DT>(d[j], a);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot[j] = __builtin_fmaf(g[i], a[i], dot[j]);
          o[i] = f[j] * g[i];
        }
        __builtin_nontemporal_store(round8<DT>(o), dD + static_cast<int64_t>(r[j]) * vecs + v);
      }
    }
    float sum = 0.0f;  // of row j0 + sub, in the token's first threads
    if constexpr (LANES < kRowThreads) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dot[j] = lanes_sum<LANES>(dot[j]);
        sum = sub == j ? dot[j] : sum;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dot[j] = wave_sum(dot[j]);
        if ((threadIdx.x & 63) == 0) sums[turn][threadIdx.x >> 6][j] = dot[j];
      }
      __syncthreads();
      sum = sums[turn][0][sub & 3];
#pragma unroll
      for (int i = 1; i < kRowThreads / 64; ++i) sum += sums[turn][i][sub & 3];
    }
    if (there && sub < 4 && j0 + sub < k) dw[t * k + j0 + sub] = sum;
  }
}

dim3 token_grid(int64_t T, int64_t vecs, int log2_threads) {
  const int64_t tokens = kRowThreads >> log2_threads, per = int64_t{1} << log2_threads;
  return dim3(static_cast<unsigned>((T + tokens - 1) / tokens), static_cast<unsigned>((vecs + per - 1) / per));
}

}  // namespace

hipError_t launch_route_gather(const void *X, const float *scale, const int *pos, void *Xs, float *scales, int64_t T,
                               int64_t rows, int vecs, int per_row, int k, hipStream_t stream) {
  const int n = token_threads_log2(vecs);
  hipLaunchKernelGGL(gather_kernel, token_grid(T, vecs, n), dim3(kRowThreads), 0, stream, static_cast<const uint4_v *>(X), scale,
                     pos, static_cast<uint4_v *>(Xs), scales, T, rows, vecs, per_row, k, n);
  return hipGetLastError();
}

hipError_t launch_route_combine(int dtype, const void *D, const int *pos, const float *w, void *Y, int64_t T, int64_t rows,
                                int vecs, int k, hipStream_t stream) {
  const int n = token_threads_log2(vecs);
  const auto kernel = dtype == kBF16 ? combine_kernel<kBF16> : combine_kernel<kF16>;
  hipLaunchKernelGGL(kernel, token_grid(T, vecs, n), dim3(kRowThreads), 0, stream, static_cast<const uint4_v *>(D), pos, w,
                     static_cast<uint4_v *>(Y), T, rows, vecs, k, n);
  return hipGetLastError();
}

// Threads of a token: rows of up to 512 numbers are a wave's or less (4096 x 8 rows of
// 512: 13.4 us, with a workgroup 14.2; 16384 x 8 of 128 13.5, 36.8; 32768 x 8 of 64 14.0, 69).
template <int DT>
hipError_t launch_combine_grad_dt(const void *dY, const void *D, const int *pos, const float *w, void *dD, float *dw, int64_t T,
                                  int64_t rows, int vecs, int k, hipStream_t stream) {
  const int lanes = vecs <= 8 ? 8 : vecs <= 16 ? 16 : vecs <= 32 ? 32 : vecs <= 64 ? 64 : kRowThreads;
  const auto kernel = lanes == 8    ? combine_grad_kernel<DT, 8>
                      : lanes == 16 ? combine_grad_kernel<DT, 16>
                      : lanes == 32 ? combine_grad_kernel<DT, 32>
                      : lanes == 64 ? combine_grad_kernel<DT, 64>
                                    : combine_grad_kernel<DT, kRowThreads>;
  const int64_t tokens = kRowThreads / lanes;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>((T + tokens - 1) / tokens)), dim3(kRowThreads), 0, stream,
                     static_cast<const uint4_v *>(dY), static_cast<const uint4_v *>(D), pos, w, static_cast<uint4_v *>(dD), dw, T,
                     rows, vecs, k);
  return hipGetLastError();
}

hipError_t launch_route_combine_grad(int dtype, const void *dY, const void *D, const int *pos, const float *w, void *dD,
                                     float *dw, int64_t T, int64_t rows, int vecs, int k, hipStream_t stream) {
  return dtype == kBF16 ? launch_combine_grad_dt<kBF16>(dY, D, pos, w, dD, dw, T, rows, vecs, k, stream)
                        : launch_combine_grad_dt<kF16>(dY, D, pos, w, dD, dw, T, rows, vecs, k, stream);
}

}  // namespace gt
