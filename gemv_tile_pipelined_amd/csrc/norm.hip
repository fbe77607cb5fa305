// norm.hip -- root-mean-square norm with the residual's addition, its output in
// 16 bits or in e4m3 with an FP32 scale for each 128 of a row, and its gradient.
//
//   h = x + residual (one rounding to 16 bits; x itself without a residual)
//   r = 1 / sqrt(mean_c(h^2) + eps)
//   y = h r weight
//
//   dx = r (weight dy) - h r^3 mean_c(weight dy h) + dh
//   dweight[c] = sum_t dy h r
//
// A workgroup holds a row in registers between the sum of squares and the output,
// so each input is read once and each output written once: bound by memory.  The
// sum of squares and r are in FP64, which costs nothing here (8192 x 4096 with the
// residual, 8 bits out, takes 46 us either way) and makes the e4m3 numbers those
// nearest to y / scale but for one in some 10^7: weight h is exact in FP32, r /
// scale has 48 bits, and the product is rounded to odd before the conversion, so
// that only real ties tie.  y in 16 bits and both gradients are FP32 until their one
// rounding.  16 lanes hold a block of 128 columns, 8 each, so a block's largest
// number is found within a lane row.
#include "fp8_common.hpp"
#include "kernels.hpp"
#include "wave_ops.hpp"

namespace gt {

namespace {

constexpr float kMinScale = 0x1p-80f;

// Sum over the workgroup, in every lane; waves are added in order.  `slots` is
// one of two buffers that the caller uses in turn, so that one barrier is enough.
template <int THREADS>
__device__ inline float group_sum(float v, float *slots) {
  v = wave_sum(v);
  if constexpr (THREADS == 64) return v;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  float sum = slots[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) sum += slots[w];
  return sum;
}

// The same in FP64.
template <int THREADS>
__device__ inline double group_sum(double v, double *slots) {
  v = wave_sum_last(v);
  if ((threadIdx.x & 63) == 63) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  double sum = slots[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) sum += slots[w];
  return sum;
}

// 1 / sqrt(v): the instruction's approximation and two Newton steps; 0, infinity
// and NaN as they come.
__device__ inline double inverse_root(double v) {
  double r = __builtin_amdgcn_rsq(v);
  if (v > 0 && v < __builtin_inf()) {
    r = r * (1.5 - 0.5 * v * r * r);
    r = r * (1.5 - 0.5 * v * r * r);
  }
  return r;
}

// p (high + low) rounded to odd: the rounded product, one bit lower where it is
// above the real one, with its last bit set unless it is that.
__device__ inline float product_to_odd(float p, float high, float low) {
  const float q = p * high;
  const float rest = __builtin_fmaf(p, low, __builtin_fmaf(p, high, -q));
  const float r = q < 0.0f ? -rest : rest;  // towards larger magnitudes
  uint32_t b = __builtin_bit_cast(uint32_t, q);
  b -= r < 0.0f ? 1u : 0u;
  b |= r != 0.0f ? 1u : 0u;
  return __builtin_bit_cast(float, b);
}

// h may be x or residual: a row's vectors are all read by the threads that write
// them, before they do.
template <int DT, int THREADS, int NV, bool FP8>
__global__ void __launch_bounds__(THREADS)
rmsnorm_kernel(const uint16_t *x, const uint16_t *residual, const uint16_t *__restrict__ weight, uint16_t *h,
               uint16_t *__restrict__ y, uint8_t *__restrict__ q, float *__restrict__ scale, float *__restrict__ rstd, int T,
               int C, float eps) {
  __shared__ double slots[2][THREADS / 64];
  const int vecs = C / 8, blocks = (C + kScaleBlock - 1) / kScaleBlock;
  const double inv_c = 1.0 / static_cast<double>(C);
  uint4_v wv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * THREADS + threadIdx.x;
    wv[i] = v < vecs ? reinterpret_cast<const uint4_v *>(weight)[v] : uint4_v{0, 0, 0, 0};
  }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x, turn ^= 1) {
    const uint4_v *xr = reinterpret_cast<const uint4_v *>(x + row * C);
    uint4_v hv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * THREADS + threadIdx.x;
      hv[i] = v < vecs ? xr[v] : uint4_v{0, 0, 0, 0};
    }
    if (residual != nullptr) {
      const uint4_v *rr = reinterpret_cast<const uint4_v *>(residual + row * C);
      uint4_v *hr = reinterpret_cast<uint4_v *>(h + row * C);
      uint4_v rv[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * THREADS + threadIdx.x;
        rv[i] = v < vecs ? rr[v] : uint4_v{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * THREADS + threadIdx.x;
        float a[8], b[8];
        widen8<DT>(hv[i], a);
        widen8<DT>(rv[i], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] += b[j];
        hv[i] = round8<DT>(a);
        if (v < vecs) hr[v] = hv[i];
      }
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8];
      widen8<DT>(hv[i], a);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fma(static_cast<double>(a[j]), static_cast<double>(a[j]), sum);
    }
    sum = group_sum<THREADS>(sum, slots[turn]);
    const double rd = inverse_root(sum * inv_c + static_cast<double>(eps));
    const float r = static_cast<float>(rd);
    if (rstd != nullptr && threadIdx.x == 0) rstd[row] = r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * THREADS + threadIdx.x;
      float a[8], w[8];
      widen8<DT>(hv[i], a);
      widen8<DT>(wv[i], w);
      if (y != nullptr) {
        float out[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          out[j] = a[j] * r * w[j];
          // y is an FP32 number in every variant: not a product that v_fma_mix*
          // rounds to half precision with it.
          asm volatile("" : "+v"(out[j]));
        }
        if (v < vecs) reinterpret_cast<uint4_v *>(y + row * C)[v] = round8<DT>(out);
      }
      if constexpr (FP8) {
        uint32_t top = 0;  // of |weight h|, as bits: NaN above infinity above the rest
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j] *= w[j];
          const uint32_t bits = __builtin_bit_cast(uint32_t, a[j]) & 0x7fffffffu;
          top = bits > top ? bits : top;
        }
        const double amax = static_cast<double>(__builtin_bit_cast(float, max_of_16_lanes(top)));
        float s = static_cast<float>(amax * rd * (1.0 / 448.0));
        s = s < kMinScale ? kMinScale : s;  // a NaN stays
        const double t = rd / static_cast<double>(s);
        const float high = static_cast<float>(t), low = static_cast<float>(t - static_cast<double>(high));
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = product_to_odd(a[j], high, low);
        int q0 = __builtin_amdgcn_cvt_pk_fp8_f32(a[0], a[1], 0, false);
        q0 = __builtin_amdgcn_cvt_pk_fp8_f32(a[2], a[3], q0, true);
        int q1 = __builtin_amdgcn_cvt_pk_fp8_f32(a[4], a[5], 0, false);
        q1 = __builtin_amdgcn_cvt_pk_fp8_f32(a[6], a[7], q1, true);
        if (v < vecs) {
          reinterpret_cast<uint2_v *>(q + row * C)[v] = uint2_v{static_cast<uint32_t>(q0), static_cast<uint32_t>(q1)};
          if ((threadIdx.x & 15) == 0) scale[row * blocks + v / 16] = s;
        }
      }
    }
  }
}

// Rows of a workgroup follow one another by the grid; a thread keeps its
// columns' share of dweight in registers over them and leaves it in `partial`
// [gridDim.x, C].  8191 x 2048 with dh: 29.7 us with the sum of the partial rows, of
// which 25.3 are its bytes at a large copy's rate.
template <int DT, int THREADS, int NV>
__global__ void __launch_bounds__(THREADS)
rmsnorm_grad_kernel(const uint16_t *__restrict__ dy, const uint16_t *__restrict__ dh, const uint16_t *__restrict__ h,
                    const uint16_t *__restrict__ weight, const float *__restrict__ rstd, uint16_t *__restrict__ dx,
                    float *__restrict__ partial, int T, int C) {
  __shared__ float slots[2][THREADS / 64];
  const int vecs = C / 8;
  const float inv_c = 1.0f / static_cast<float>(C);
  uint4_v wv[NV];
  float dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * THREADS + threadIdx.x;
    wv[i] = v < vecs ? reinterpret_cast<const uint4_v *>(weight)[v] : uint4_v{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x, turn ^= 1) {
    const float r = rstd[row];
    uint4_v dv[NV], hv[NV], ev[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * THREADS + threadIdx.x;
      const bool in = v < vecs;
      dv[i] = in ? reinterpret_cast<const uint4_v *>(dy + row * C)[v] : uint4_v{0, 0, 0, 0};
      hv[i] = in ? reinterpret_cast<const uint4_v *>(h + row * C)[v] : uint4_v{0, 0, 0, 0};
      ev[i] = in && dh != nullptr ? reinterpret_cast<const uint4_v *>(dh + row * C)[v] : uint4_v{0, 0, 0, 0};
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8], b[8], w[8];
      widen8<DT>(dv[i], a);
      widen8<DT>(hv[i], b);
      widen8<DT>(wv[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = b[j] * r;
        dw[i][j] = __builtin_fmaf(a[j], n, dw[i][j]);
        dot = __builtin_fmaf(a[j] * w[j], n, dot);
      }
    }
    dot = group_sum<THREADS>(dot, slots[turn]) * inv_c;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * THREADS + threadIdx.x;
      float a[8], b[8], w[8], e[8];
      widen8<DT>(dv[i], a);
      widen8<DT>(hv[i], b);
      widen8<DT>(wv[i], w);
      widen8<DT>(ev[i], e);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = __builtin_fmaf(r, __builtin_fmaf(-(b[j] * r), dot, a[j] * w[j]), e[j]);
      if (v < vecs) reinterpret_cast<uint4_v *>(dx + row * C)[v] = round8<DT>(a);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * THREADS + threadIdx.x;
    if (v < vecs) {
      float4_t *out = reinterpret_cast<float4_t *>(partial + static_cast<int64_t>(blockIdx.x) * C + 8 * v);
      out[0] = float4_t{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
      out[1] = float4_t{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
  }
}

// dweight[c] = the sum of `parts` rows of partial [parts, C]: 32 columns to a
// workgroup, 32 threads to a column, each a run of rows whose loads are in flight
// together (8 threads to a column: 8191 x 2048 in 31.2 us in all, not 29.7).
constexpr int kReduceCols = 32, kReduceRuns = 32;
__global__ void __launch_bounds__(kReduceCols *kReduceRuns)
rmsnorm_reduce_kernel(const float *__restrict__ partial, float *__restrict__ dweight, int parts, int C) {
  __shared__ float sums[kReduceRuns][kReduceCols];
  const int col = static_cast<int>(blockIdx.x) * kReduceCols + (threadIdx.x & (kReduceCols - 1));
  const int run = threadIdx.x / kReduceCols;
  float sum = 0.0f;
  if (col < C) {
    const int end = (run + 1) * parts / kReduceRuns;
#pragma unroll 16
    for (int p = run * parts / kReduceRuns; p < end; ++p) sum += partial[static_cast<int64_t>(p) * C + col];
  }
  sums[run][threadIdx.x & (kReduceCols - 1)] = sum;
  __syncthreads();
  if (run == 0 && col < C) {
#pragma unroll
    for (int i = 1; i < kReduceRuns; ++i) sum += sums[i][threadIdx.x];
    dweight[col] = sum;
  }
}

// Workgroups of the norm at most; each then takes several rows.  8192 x 4096: 46.5 us
// with 256 threads, with 2048 workgroups and with one for each row; with 512 threads
// 48.3 and 46.3 to 48.
constexpr int kNormGrid = 16384;

template <int DT, int THREADS, int NV>
hipError_t launch_norm(const NormArgs &a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.T < kNormGrid ? a.T : kNormGrid));
  const auto kernel = a.q != nullptr ? rmsnorm_kernel<DT, THREADS, NV, true> : rmsnorm_kernel<DT, THREADS, NV, false>;
  hipLaunchKernelGGL(kernel, grid, dim3(THREADS), 0, stream, static_cast<const uint16_t *>(a.x),
                     static_cast<const uint16_t *>(a.residual), static_cast<const uint16_t *>(a.weight),
                     static_cast<uint16_t *>(a.h), static_cast<uint16_t *>(a.y), static_cast<uint8_t *>(a.q), a.scale, a.rstd,
                     a.T, a.C, a.eps);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_norm_dt(const NormArgs &a, hipStream_t stream) {
  const int vecs = a.C / 8;
  if (vecs <= 64) return launch_norm<DT, 64, 1>(a, stream);
  if (vecs <= 128) return launch_norm<DT, 128, 1>(a, stream);
  if (vecs <= 256) return launch_norm<DT, 256, 1>(a, stream);
  if (vecs <= 512) return launch_norm<DT, 256, 2>(a, stream);
  if (vecs <= 1024) return launch_norm<DT, 512, 2>(a, stream);
  if (vecs <= 2048) return launch_norm<DT, 512, 4>(a, stream);
  return launch_norm<DT, 1024, 4>(a, stream);
}

template <int DT, int THREADS, int NV>
hipError_t launch_grad(const NormGradArgs &a, hipStream_t stream) {
  const int parts = rmsnorm_grad_parts(a.T);
  if (parts > 0) {  // without rows dweight is a sum of nothing
    hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, THREADS, NV>), dim3(parts), dim3(THREADS), 0, stream,
                       static_cast<const uint16_t *>(a.dy), static_cast<const uint16_t *>(a.dh),
                       static_cast<const uint16_t *>(a.h), static_cast<const uint16_t *>(a.weight), a.rstd,
                       static_cast<uint16_t *>(a.dx), a.workspace, a.T, a.C);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(rmsnorm_reduce_kernel, dim3((a.C + kReduceCols - 1) / kReduceCols), dim3(kReduceCols * kReduceRuns), 0,
                     stream, a.workspace, a.dweight, parts, a.C);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_grad_dt(const NormGradArgs &a, hipStream_t stream) {
  const int vecs = a.C / 8;
  if (vecs <= 64) return launch_grad<DT, 64, 1>(a, stream);
  if (vecs <= 128) return launch_grad<DT, 128, 1>(a, stream);
  if (vecs <= 256) return launch_grad<DT, 256, 1>(a, stream);
  if (vecs <= 512) return launch_grad<DT, 512, 1>(a, stream);
  if (vecs <= 1024) return launch_grad<DT, 512, 2>(a, stream);
  if (vecs <= 2048) return launch_grad<DT, 512, 4>(a, stream);
  return launch_grad<DT, 1024, 4>(a, stream);
}

}  // namespace

hipError_t launch_rmsnorm(int dtype, const NormArgs &a, hipStream_t stream) {
  return dtype == kBF16 ? launch_norm_dt<kBF16>(a, stream) : launch_norm_dt<kF16>(a, stream);
}

int rmsnorm_grad_parts(int64_t T) { return static_cast<int>(T < 512 ? T : 512); }

hipError_t launch_rmsnorm_grad(int dtype, const NormGradArgs &a, hipStream_t stream) {
  return dtype == kBF16 ? launch_grad_dt<kBF16>(a, stream) : launch_grad_dt<kF16>(a, stream);
}

}  // namespace gt
