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
// A row is held in registers between the sum of squares and the output, so each input
// is read once and each output written once: bound by memory.  Rows of up to 1536
// columns are a wave's or less, several to a workgroup, and need no barrier; longer
// ones are a workgroup's.  eps, the sum of squares and r are in FP64, which costs nothing
// here (8192 x 4096 with the residual, 8 bits out, takes 46 us either way) and makes the
// e4m3 numbers those nearest to y / scale: weight h is exact in FP32, r / scale has 48
// bits, and the product is rounded to odd before the conversion, so that nothing ties that
// is further than 2^-47 of itself from the middle of two.  y in 16 bits and both gradients
// are FP32 until their one rounding.  16 lanes hold a block of 128 columns, 8 each, so a
// block's largest number is found within a lane row.
#include "fp8_common.hpp"
#include "kernels.hpp"
#include "wave_ops.hpp"

namespace gt {

namespace {

constexpr float kMinScale = 0x1p-80f;

// Which of a workgroup's ROWS rows this thread is at; the same for a whole wave if the
// row has one.
template <int LANES, int ROWS>
__device__ inline int row_group() {
  if constexpr (ROWS == 1) return 0;
  const int group = static_cast<int>(threadIdx.x) / LANES;
  if constexpr (LANES < 64) return group;
  return __builtin_amdgcn_readfirstlane(group);
}

// Sum over the LANES threads of a row, in every one of them: within a wave, or over
// the waves of a workgroup (LANES > 64, one row a workgroup), added in order.  `slots`
// is one of two buffers that the caller uses in turn, so that one barrier is enough.
template <int LANES>
__device__ inline float row_sum(float v, float *slots) {
  if constexpr (LANES <= 64) return lanes_sum<LANES>(v);
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  float sum = slots[0];
#pragma unroll
  for (int w = 1; w < LANES / 64; ++w) sum += slots[w];
  return sum;
}

// The same in FP64.
template <int LANES>
__device__ inline double row_sum(double v, double *slots) {
  if constexpr (LANES <= 64) return lanes_sum<LANES>(v);
  v = wave_sum_last(v);
  if ((threadIdx.x & 63) == 63) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  double sum = slots[0];
#pragma unroll
  for (int w = 1; w < LANES / 64; ++w) sum += slots[w];
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

// p (high + low), high > 0, rounded to odd: the rounded product, one bit lower where it
// is above the real one, with its last bit set unless it is that.  `low` is in the product
// before it is rounded: p high alone can be more than a unit off, and one bit lower is
// then still above.  Magnitudes, and p's sign: that of a zero is kept.
__device__ inline float product_to_odd(float p, float high, float low) {
  const float a = __builtin_fabsf(p);
  const float q = __builtin_fmaf(a, high, a * low);
  const float rest = __builtin_fmaf(a, low, __builtin_fmaf(a, high, -q));
  uint32_t b = __builtin_bit_cast(uint32_t, q);
  b -= rest < 0.0f ? 1u : 0u;
  b |= rest != 0.0f ? 1u : 0u;
  return __builtin_copysignf(__builtin_bit_cast(float, b), p);
}

// Rows whose r is outside this are multiplied in FP64: below, it is no normal FP32 number;
// above, a product weight h that FP32 does not hold exactly (below 2^-134) may stand for
// more than a zero of e4m3 (2^-90 and less).  So are blocks whose largest weight h is 2^100
// or more: it may leave FP32's range, as y need not, and the lower half of r / scale would
// be below the normal numbers.
constexpr double kLeastRoot = 0x1p-126, kMostRoot = 0x1p40;
constexpr uint32_t kLargeProduct = 0x71800000;  // 2^100, as bits
// The power of two that brings r to 2^36 .. 2^37, and weight h r 2^-that, of which 2^-90 to
// 2^136 matter, to 2^-127 and more (16 bits of it are exact there) and 2^100 and less.
__device__ inline int root_exponent(double r) {
  return r == 0.0 ? -300 : r < __builtin_inf() ? __builtin_amdgcn_frexp_exp(r) - 37 : 0;
}

// A number in FP64, converted where it is needed: the compiler would otherwise keep those
// of the sum of squares, and of the weight over all rows, in registers for it.
__device__ inline double afresh(float v) {
  asm volatile("" : "+v"(v));
  return static_cast<double>(v);
}

// h may be x or residual: a row's vectors are all read by the threads that write
// them, before they do.
template <int DT, int LANES, int NV, int ROWS, bool FP8>
__global__ void __launch_bounds__(LANES *ROWS)
rmsnorm_kernel(const uint16_t *x, const uint16_t *residual, const uint16_t *__restrict__ weight, uint16_t *h,
               uint16_t *__restrict__ y, uint8_t *__restrict__ q, float *__restrict__ scale, float *__restrict__ rstd, int T,
               int C, double eps) {
  __shared__ double slots[2][(LANES + 63) / 64];
  const int group = row_group<LANES, ROWS>(), sub = static_cast<int>(threadIdx.x) - group * LANES;
  const int vecs = C / 8, blocks = (C + kScaleBlock - 1) / kScaleBlock;
  const double inv_c = 1.0 / static_cast<double>(C);
  uint4_v wv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * LANES + sub;
    wv[i] = v < vecs ? reinterpret_cast<const uint4_v *>(weight)[v] : uint4_v{0, 0, 0, 0};
  }
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + group; row < T;
       row += static_cast<int64_t>(gridDim.x) * ROWS, turn ^= 1) {
    const uint4_v *xr = reinterpret_cast<const uint4_v *>(x + row * C);
    uint4_v hv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * LANES + sub;
      hv[i] = v < vecs ? xr[v] : uint4_v{0, 0, 0, 0};
    }
    if (residual != nullptr) {
      const uint4_v *rr = reinterpret_cast<const uint4_v *>(residual + row * C);
      uint4_v *hr = reinterpret_cast<uint4_v *>(h + row * C);
      uint4_v rv[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * LANES + sub;
        rv[i] = v < vecs ? rr[v] : uint4_v{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * LANES + sub;
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
    sum = row_sum<LANES>(sum, slots[turn]);
    const double rd = inverse_root(sum * inv_c + eps);
    const float r = static_cast<float>(rd);
    if (rstd != nullptr && sub == 0) rstd[row] = r;
    const bool far = !(rd >= kLeastRoot && rd <= kMostRoot);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * LANES + sub;
      float a[8], w[8];
      widen8<DT>(hv[i], a);
      widen8<DT>(wv[i], w);
      if (y != nullptr) {
        float out[8];
        if (__builtin_expect(far, 0)) {
#pragma unroll
          for (int j = 0; j < 8; ++j) out[j] = static_cast<float>(afresh(a[j]) * rd * afresh(w[j]));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) out[j] = a[j] * r * w[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // y is an FP32 number in every variant: not a product that v_fma_mix*
          // rounds to half precision with it.
          asm volatile("" : "+v"(out[j]));
        }
        if (v < vecs) reinterpret_cast<uint4_v *>(y + row * C)[v] = round8<DT>(out);
      }
      if constexpr (FP8) {
        const auto block_max = [&] {  // as bits: NaN above infinity above the rest
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t bits = __builtin_bit_cast(uint32_t, a[j]) & 0x7fffffffu;
            top = bits > top ? bits : top;
          }
          return LANES == 8 ? max_of_8_lanes(top) : max_of_16_lanes(top);
        };
        double root = rd;  // y is a[] times root
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] *= w[j];
        uint32_t top = block_max();
        if (__builtin_expect(far || top >= kLargeProduct, 0)) {  // a block's lanes alike
          const int e = root_exponent(rd);
          root = __builtin_ldexp(rd, -e);
          widen8<DT>(hv[i], a);
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] = static_cast<float>(__builtin_ldexp(afresh(a[j]) * afresh(w[j]), e));
          top = block_max();
        }
        float s = static_cast<float>(static_cast<double>(__builtin_bit_cast(float, top)) * root * (1.0 / 448.0));
        s = s < kMinScale ? kMinScale : s;  // a NaN stays
        const double t = root / static_cast<double>(s);
        const float high = static_cast<float>(t), low = static_cast<float>(t - static_cast<double>(high));
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = product_to_odd(a[j], high, low);
        int q0 = __builtin_amdgcn_cvt_pk_fp8_f32(a[0], a[1], 0, false);
        q0 = __builtin_amdgcn_cvt_pk_fp8_f32(a[2], a[3], q0, true);
        int q1 = __builtin_amdgcn_cvt_pk_fp8_f32(a[4], a[5], 0, false);
        q1 = __builtin_amdgcn_cvt_pk_fp8_f32(a[6], a[7], q1, true);
        if (v < vecs) {
          reinterpret_cast<uint2_v *>(q + row * C)[v] = uint2_v{static_cast<uint32_t>(q0), static_cast<uint32_t>(q1)};
          if ((sub & 15) == 0) scale[row * blocks + v / 16] = s;
        }
      }
    }
  }
}

// Rows of a workgroup follow one another by the grid; a thread keeps its columns'
// share of dweight in registers over them (in LDS, in places of its own, where the
// registers do not hold it) and leaves it in `partial` [gridDim.x, C].  AHEAD: the next
// row is on its way while this one is worked on, for rows of which a CU has only one.
// 8191 x 2048 with dh: 29.7 us with the sum of the partial rows, of which 25.3 are its
// bytes at a large copy's rate.
template <int DT, int LANES, int NV, int ROWS, bool AHEAD>
__global__ void __launch_bounds__(LANES *ROWS)
rmsnorm_grad_kernel(const uint16_t *__restrict__ dy, const uint16_t *__restrict__ dh, const uint16_t *__restrict__ h,
                    const uint16_t *__restrict__ weight, const float *__restrict__ rstd, uint16_t *__restrict__ dx,
                    float *__restrict__ partial, int T, int C) {
  __shared__ float slots[2][(LANES + 63) / 64];
  const int group = row_group<LANES, ROWS>(), sub = static_cast<int>(threadIdx.x) - group * LANES;
  const int vecs = C / 8;
  const float inv_c = 1.0f / static_cast<float>(C);
  constexpr bool kFar = LANES * NV > 2048;  // dw is in LDS, and dh is read late
  __shared__ float4_t far[kFar ? 2 * LANES * NV : 1];
  uint4_v wv[NV], dv[NV], hv[NV], ev[NV];
  float dw[NV][8], r = 0.0f;
  const auto load = [&](const uint4_v *src, uint4_v (&to)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * LANES + sub;
      to[i] = src != nullptr && v < vecs ? src[v] : uint4_v{0, 0, 0, 0};
    }
  };
  const auto row_of = [&](const uint16_t *p, int64_t row) {
    return p != nullptr ? reinterpret_cast<const uint4_v *>(p + row * C) : nullptr;
  };
  const auto load_row = [&](int64_t row, uint4_v (&d)[NV], uint4_v (&hh)[NV], uint4_v (&e)[NV], float &rr) {
    rr = rstd[row];
    load(row_of(dy, row), d);
    load(row_of(h, row), hh);
    if constexpr (!kFar) load(row_of(dh, row), e);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  if constexpr (kFar) {
#pragma unroll
    for (int i = 0; i < 2 * NV; ++i) far[i * LANES + sub] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  load(reinterpret_cast<const uint4_v *>(weight), wv);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + group, step = static_cast<int64_t>(gridDim.x) * ROWS;
  uint4_v dn[NV], hn[NV], en[NV];
  float rn = 0.0f;
  if (AHEAD && first < T) load_row(first, dn, hn, en, rn);
  int turn = 0;
  for (int64_t row = first; row < T; row += step, turn ^= 1) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        dv[i] = dn[i];
        hv[i] = hn[i];
        ev[i] = en[i];
      }
      r = rn;
      if (row + step < T) load_row(row + step, dn, hn, en, rn);
    } else {
      load_row(row, dv, hv, ev, r);
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8], b[8], w[8];
      widen8<DT>(dv[i], a);
      widen8<DT>(hv[i], b);
      widen8<DT>(wv[i], w);
      float4_t lo, hi;
      if constexpr (kFar) {
        lo = far[2 * i * LANES + sub];
        hi = far[(2 * i + 1) * LANES + sub];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = b[j] * r;
        if constexpr (!kFar) dw[i][j] = __builtin_fmaf(a[j], n, dw[i][j]);
        else if (j < 4) lo[j] = __builtin_fmaf(a[j], n, lo[j]);
        else hi[j - 4] = __builtin_fmaf(a[j], n, hi[j - 4]);
        dot = __builtin_fmaf(a[j] * w[j], n, dot);
      }
      if constexpr (kFar) {
        far[2 * i * LANES + sub] = lo;
        far[(2 * i + 1) * LANES + sub] = hi;
      }
    }
    dot = row_sum<LANES>(dot, slots[turn]) * inv_c;
    if constexpr (kFar) load(row_of(dh, row), ev);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * LANES + sub;
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
  if constexpr (ROWS > 1) {
    // The shares of the rows that went side by side, in their order.
    __shared__ __attribute__((aligned(16))) float sums[ROWS][LANES * NV * 8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float4_t *to = reinterpret_cast<float4_t *>(&sums[group][(i * LANES + sub) * 8]);
      to[0] = float4_t{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
      to[1] = float4_t{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += LANES * ROWS) {
      float sum = sums[0][c];
#pragma unroll
      for (int r = 1; r < ROWS; ++r) sum += sums[r][c];
      partial[static_cast<int64_t>(blockIdx.x) * C + c] = sum;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * LANES + sub;
      if (v < vecs) {
        typedef float float4_u __attribute__((ext_vector_type(4), aligned(4)));  // dweight itself is 4-byte aligned
        float4_u *out = reinterpret_cast<float4_u *>(partial + static_cast<int64_t>(blockIdx.x) * C + 8 * v);
        out[0] = kFar ? far[2 * i * LANES + sub] : float4_t{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
        out[1] = kFar ? far[(2 * i + 1) * LANES + sub] : float4_t{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
      }
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
// Workgroups of the gradient at most, each with a row of partial sums; half as many for
// long rows, whose partial sums are bytes that count.  The workspace has room for
// kNormParts of them, or one for each row, whatever the columns.
constexpr int kNormParts = 512, kLongRowParts = 256;

template <int DT, int LANES, int NV, int ROWS = 1>
hipError_t launch_norm(const NormArgs &a, hipStream_t stream) {
  const int blocks = (a.T + ROWS - 1) / ROWS;
  const dim3 grid(static_cast<unsigned>(blocks < kNormGrid ? blocks : kNormGrid));
  const auto kernel = a.q != nullptr ? rmsnorm_kernel<DT, LANES, NV, ROWS, true> : rmsnorm_kernel<DT, LANES, NV, ROWS, false>;
  hipLaunchKernelGGL(kernel, grid, dim3(LANES * ROWS), 0, stream, static_cast<const uint16_t *>(a.x),
                     static_cast<const uint16_t *>(a.residual), static_cast<const uint16_t *>(a.weight),
                     static_cast<uint16_t *>(a.h), static_cast<uint16_t *>(a.y), static_cast<uint8_t *>(a.q), a.scale, a.rstd,
                     a.T, a.C, a.eps);
  return hipGetLastError();
}

// LANES, NV, ROWS for a row's pieces of 8 columns.  2^25 numbers, us without a residual /
// with it / with 8 bits out (bytes at a large copy's rate: 25.3, 50.6, 44.3): C = 64 29 / 48 /
// 47 (a wave a row 95 / 147 / 207), 128 27 / 48 / 48 (54 / 85 / 110), 256 26 / 48 / 47 (33 / 55 /
// 62), 1024 25 / 48 / 46 (two waves a row 26 / 51 / 47), 1536 25 / 48 / 47 (four 30 / 49 / 49), 2048
// 27 / 48 / 47 (a wave a row 25 / 47 / 47), 20480 30 / 57 / 62 (four pieces a thread 30 / 59 / 64).
template <int DT>
hipError_t launch_norm_dt(const NormArgs &a, hipStream_t stream) {
  const int vecs = a.C / 8;
  if (vecs <= 8) return launch_norm<DT, 8, 1, 32>(a, stream);
  if (vecs <= 16) return launch_norm<DT, 16, 1, 16>(a, stream);
  if (vecs <= 32) return launch_norm<DT, 32, 1, 8>(a, stream);
  if (vecs <= 64) return launch_norm<DT, 64, 1, 4>(a, stream);
  if (vecs <= 128) return launch_norm<DT, 64, 2, 4>(a, stream);
  if (vecs <= 192) return launch_norm<DT, 64, 3, 4>(a, stream);
  if (vecs <= 256) return launch_norm<DT, 256, 1>(a, stream);
  if (vecs <= 512) return launch_norm<DT, 256, 2>(a, stream);
  if (vecs <= 1024) return launch_norm<DT, 512, 2>(a, stream);
  if (vecs <= 2048) return launch_norm<DT, 512, 4>(a, stream);
  if (vecs <= 3 * 1024) return launch_norm<DT, 1024, 3>(a, stream);
  return launch_norm<DT, 1024, 4>(a, stream);
}

template <int DT, int LANES, int NV, int ROWS = 1, int PARTS = kNormParts, bool AHEAD = false>
hipError_t launch_grad(const NormGradArgs &a, hipStream_t stream) {
  // Few rows are one workgroup's, whose partial sums are the result: one launch
  // (us with one / two: 1 x 4096 2.6 / 4.7, 2 x 4096 3.2 / 4.9, 8 x 512 2.9 / 4.4, 64 x 64 3.0 / 4.4,
  // 2 x 32768 13.1 / 12.3).
  static_assert(PARTS <= kNormParts && ROWS >= 1, "the partial sums fit rmsnorm_grad_parts rows");
  const int rounds = (a.T + ROWS - 1) / ROWS;
  const int parts = rounds <= 2 ? (rounds > 0 ? 1 : 0) : rounds < PARTS ? rounds : PARTS;
  if (parts > 0) {  // without rows dweight is a sum of nothing
    hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, LANES, NV, ROWS, AHEAD>), dim3(parts), dim3(LANES * ROWS), 0, stream,
                       static_cast<const uint16_t *>(a.dy), static_cast<const uint16_t *>(a.dh),
                       static_cast<const uint16_t *>(a.h), static_cast<const uint16_t *>(a.weight), a.rstd,
                       static_cast<uint16_t *>(a.dx), parts == 1 ? a.dweight : a.workspace, a.T, a.C);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || parts == 1) return e;
  }
  hipLaunchKernelGGL(rmsnorm_reduce_kernel, dim3((a.C + kReduceCols - 1) / kReduceCols), dim3(kReduceCols * kReduceRuns), 0,
                     stream, a.workspace, a.dweight, parts, a.C);
  return hipGetLastError();
}

// As above.  2^25 numbers with dh, us (bytes 50.6): C = 64 51 (a wave a row, one to a
// workgroup: 778), 128 52 (389), 512 51 (120), 1024 53 (two waves a row 76), 1536 54 (four 60),
// 2048 53 (a wave a row 54), 5120 55 (512 threads and workgroups, not AHEAD 56), 8192 55 (57),
// 12288 58 (63), 16384 60 (67; AHEAD does not fit the registers: 118), 20480 62 (1024 threads of
// 4 pieces, dw in registers that it does not have, 277; 512 of 6 67), 32768 74 (220; 1024 of 4 80).
template <int DT>
hipError_t launch_grad_dt(const NormGradArgs &a, hipStream_t stream) {
  const int vecs = a.C / 8;
  if (vecs <= 8) return launch_grad<DT, 8, 1, 32>(a, stream);
  if (vecs <= 16) return launch_grad<DT, 16, 1, 16>(a, stream);
  if (vecs <= 32) return launch_grad<DT, 32, 1, 8>(a, stream);
  if (vecs <= 64) return launch_grad<DT, 64, 1, 4>(a, stream);
  if (vecs <= 128) return launch_grad<DT, 64, 2, 4>(a, stream);
  if (vecs <= 192) return launch_grad<DT, 64, 3, 4>(a, stream);
  if (vecs <= 256) return launch_grad<DT, 256, 1>(a, stream);
  if (vecs <= 512) return launch_grad<DT, 512, 1>(a, stream);
  if (vecs <= 1024) return launch_grad<DT, 1024, 1, 1, kLongRowParts, true>(a, stream);
  if (vecs <= 2048) return launch_grad<DT, 1024, 2, 1, kLongRowParts>(a, stream);
  if (vecs <= 3 * 1024) return launch_grad<DT, 1024, 3, 1, kLongRowParts>(a, stream);
  return launch_grad<DT, 512, 8, 1, kLongRowParts>(a, stream);
}

}  // namespace

hipError_t launch_rmsnorm(int dtype, const NormArgs &a, hipStream_t stream) {
  return dtype == kBF16 ? launch_norm_dt<kBF16>(a, stream) : launch_norm_dt<kF16>(a, stream);
}

int rmsnorm_grad_parts(int64_t T) { return static_cast<int>(T < kNormParts ? T : kNormParts); }

hipError_t launch_rmsnorm_grad(int dtype, const NormGradArgs &a, hipStream_t stream) {
  return dtype == kBF16 ? launch_grad_dt<kBF16>(a, stream) : launch_grad_dt<kF16>(a, stream);
}

}  // namespace gt
