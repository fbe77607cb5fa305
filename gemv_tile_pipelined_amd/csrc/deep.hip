// deep.hip -- products with fewer tiles than CUs: dense ones of block-scaled
// e4m3 operands (fp8_gemm.hip), and grouped ones of either kind
// (grouped_kernel.hpp).
//
// Such a product is bound by latency: a CU has one tile and walks its K tiles
// one after another (128x128 outputs take 0.5 us for each, whatever M).  So
// tiles are small here, the smallest of which there are no more than CUs, and
// the waves form TEAMS teams that take K tiles (128 bytes of a row) in turn,
// each with a ring of its own; together the rings fill the LDS.  A step has one
// barrier: behind it, all waves have the team's K tile kt in registers (its
// stage is refilled) and kt + 1 has landed, whose operands are read while kt's
// products are formed.  The teams' sums are joined in LDS, in order.
//
// Measured (MI355X, us; M x 4096 x 4096 in 8 bits):
//             streamed  32x32  32x64  64x64  tiles of fp8_gemm.hip
//   M =   4        5.2    6.2    8.3    9.5   15.9
//        16        6.1    6.3                 15.9
//        17               6.2    8.2    9.7   15.9
//        64               7.1    8.6   11.1   16.3
//       128              11.8    8.7   11.0   18.8
//       256              21.5   15.9   11.3   19.0
//       512 (128x64: 18.0)                    19.2
// One team (64x64, 8 stages) 13.8 us at M = 128, four of half the depth 13.2, two
// 11.1; loads issued before a step's reads and MFMAs 11.1, between them 11.6.
// Streaming (stream.hip) reads x again for every 16 rows of W: against 4096x14336
// it takes 11.8, 13.0 and 15.9 us for M = 4, 8 and 16, and small tiles 12.0, 12.2
// and 12.4.  (28672x4096 has more 128x64 tiles than there are CUs: from M = 5 on
// it goes to fp8_gemm.hip, 28.4 and 28.5 us for M = 8 and 16; streamed 27.0 and
// 31.7, and 23.6 for M = 4, which is streamed.)
// Just past a fit the larger tile costs: 1024x1024x8192 (64x64) 18.4 us,
// 1024x1025x8192 (128x64) 31.9.
// Groups (512 uneven rows over 8, x 2048 x 4096, 128x64 tiles): 8 bits 17.4 us,
// tiles of fp8_gemm.hip 20.5; bf16 33.7, tiles of grouped_kernel.hpp 40.9.  24
// rows over 8 groups x 2048 x 2048 (32x64): 8.0 and 10.7, streamed 8.5 and 12.8.
#include "fp8_common.hpp"
#include "groups.hpp"
#include "kernels.hpp"
#include "tile_order.hpp"
#include "tile_store.hpp"

#include <type_traits>

namespace gt {

namespace {

struct DeepArgs {
  const uint8_t *A, *B;
  const float *sa, *sb;
  const int *offsets;
  uint16_t *D;
  int M, N, E;    // M: rows of A (all groups)
  int row_bytes;  // of A and B
  int tiles_m, tiles_n;
  int alignment;  // of D's rows
};

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int TEAMS_, int STAGES_>
struct DeepShape {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, TEAMS = TEAMS_, STAGES = STAGES_;
  static constexpr int kWaves = WAVES_M * WAVES_N;  // of a team
  static constexpr int kThreads = 64 * kWaves * TEAMS;
  static constexpr int kWaveM = BM / WAVES_M, kWaveN = BN / WAVES_N;
  static constexpr int kFragM = kWaveM / 16, kFragN = kWaveN / 16;
  static constexpr int kRowBytes = kScaleBlock;
  static constexpr int kRowStep = 8 * kWaves;  // rows per load of all waves
  static constexpr int kDmaA = BM / kRowStep, kDmaB = BN / kRowStep;
  static constexpr int kStageA = BM * kRowBytes;
  static constexpr int kStageScales = (BM + BN) * kRowBytes;
  // Scales of A's rows, then of B's, in whole loads of 64.
  static constexpr int kScalesA = (BM + 63) / 64 * 64;
  static constexpr int kScaleWaves = (kScalesA + BN + 63) / 64;
  static constexpr int kStageBytes = kStageScales + kWaves * 256;
  static constexpr int kPerStage = kDmaA + kDmaB + 1;
  static constexpr int kTilePitch = kWaveN * 2 + 16;
  static constexpr int kRingBytes = TEAMS * STAGES * kStageBytes;  // a ring per team
  static_assert(kWaves >= kScaleWaves && kScaleBlock % BN == 0, "64 rows' scales per wave");
  static_assert(kRowStep % 16 == 0 && BM % kRowStep == 0 && BN % kRowStep == 0, "operand loads");
  static_assert(kWaves * kWaveM * kTilePitch <= kRingBytes && kRingBytes <= 160 * 1024, "LDS");
  static_assert((STAGES - 1) * kPerStage <= 63, "vmcnt range");
  // As Fp8Shape::swz (fp8_gemm.hip).
  __host__ __device__ static constexpr int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }
};

constexpr int kE4m3 = 2;

__device__ inline int4_t half_of(int8_v v, int h) {
  return h == 0 ? __builtin_shufflevector(v, v, 0, 1, 2, 3) : __builtin_shufflevector(v, v, 4, 5, 6, 7);
}

// IN: kF16, kBF16 (16-bit operands, no scales: two MFMAs of 32 per 128 bytes) or
// kE4m3.  SB: rows of B per scale.
template <class S, int IN, int OUT, bool GROUPED, int SB>
__global__ void __launch_bounds__(S::kThreads) deep_kernel(DeepArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[S::kRingBytes];
  const int lane = threadIdx.x & 63;
  const int team = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) / S::kWaves);
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % S::kWaves);
  const int wm = wave / S::WAVES_N;
  const int wn = wave % S::WAVES_N;
  char *const ring = smem + team * (S::STAGES * S::kStageBytes);
  const uint32_t lds0 = lds_addr(smem) + static_cast<uint32_t>(team) * (S::STAGES * S::kStageBytes);
  constexpr bool kScaled = IN == kE4m3;
  const int rb = a.row_bytes;
  const int KT = (rb + S::kRowBytes - 1) / S::kRowBytes;

  GroupUnit g{0, 0, a.M};
  int n0;
  if constexpr (GROUPED) {
    // A unit's tiles side by side, spread over the XCDs.
    const int unit = static_cast<int>(blockIdx.x) / a.tiles_n;
    if (!find_unit(a.offsets, a.E, a.M, S::BM, unit, &g)) return;
    n0 = (static_cast<int>(blockIdx.x) - unit * a.tiles_n) * S::BN;
  } else {
    const TileCoord tc = tile_of(xcd_logical_id(blockIdx.x, gridDim.x), a.tiles_m, a.tiles_n, kGemmGroupM);
    g.row = static_cast<int>(tc.tm) * S::BM;
    n0 = static_cast<int>(tc.tn) * S::BN;
  }
  const int m0 = g.row;
  const int rows = min(S::BM, g.end - m0), cols = min(S::BN, a.N - n0);
  const int64_t b_row = static_cast<int64_t>(g.group) * a.N + n0;
  const int4_t rsrc_a = make_buffer_rsrc(a.A + static_cast<int64_t>(m0) * rb, static_cast<uint32_t>(rows) * rb);
  const int4_t rsrc_b = make_buffer_rsrc(a.B + b_row * rb, static_cast<uint32_t>(cols) * rb);

  const int ld_row = wave * 8 + lane / 8;
  const int ld_k = ((lane % 8) ^ S::swz(ld_row)) * 16;  // bytes
  const uint32_t ld_off = static_cast<uint32_t>(ld_row) * static_cast<uint32_t>(rb) + static_cast<uint32_t>(ld_k);
  const uint32_t ld_step = static_cast<uint32_t>(S::kRowStep) * static_cast<uint32_t>(rb);
  // Scales: wave w loads those of 64 of A's rows followed by B's; waves that
  // have none left load the first ones again, to a place that nothing reads.
  const int scale_part = wave % S::kScaleWaves;
  const bool scale_a = scale_part < S::kScalesA / 64;
  const int scale_row = (scale_a ? scale_part : scale_part - S::kScalesA / 64) * 64 + lane;
  const uint32_t scale_off =
      static_cast<uint32_t>(scale_a || SB == 1 ? scale_row : scale_row / kScaleBlock) * static_cast<uint32_t>(KT) * 4u;
  int4_t rsrc_s{};
  if constexpr (kScaled) {
    const int64_t sb_row = SB == 1 ? b_row
                                   : static_cast<int64_t>(g.group) * ((a.N + kScaleBlock - 1) / kScaleBlock) + n0 / kScaleBlock;
    const int sb_rows = SB == 1 ? cols : 1;
    rsrc_s = make_buffer_rsrc(scale_a ? a.sa + static_cast<int64_t>(m0) * KT : a.sb + sb_row * KT,
                              static_cast<uint32_t>(scale_a ? rows : sb_rows) * KT * 4u);
  }
  // K tiles past the last: operands out of range, i.e. zeros, and scales of
  // another row or out of range, which belong to sums that nothing uses.
  // kt: the team's own count.
  auto issue = [&](int own, int slot) {
    const int kt = own * S::TEAMS + team;
    const uint32_t stage = lds0 + static_cast<uint32_t>(slot) * S::kStageBytes;
    const int k0 = kt * S::kRowBytes;
    const uint32_t off = k0 + ld_k < rb ? ld_off + static_cast<uint32_t>(k0) : kOobOffset;
#pragma unroll
    for (int d = 0; d < S::kDmaA + S::kDmaB; ++d) {
      const bool is_a = d < S::kDmaA;
      const int i = is_a ? d : d - S::kDmaA;
      lds_dma_b128(is_a ? rsrc_a : rsrc_b, off + i * ld_step,
                   __builtin_amdgcn_readfirstlane(stage + (is_a ? 0 : S::kStageA) + (i * S::kWaves + wave) * 1024));
    }
    if constexpr (kScaled)
      lds_dma_b32(rsrc_s, kt < KT ? scale_off + static_cast<uint32_t>(kt) * 4u : kOobOffset,
                  __builtin_amdgcn_readfirstlane(stage + S::kStageScales + static_cast<uint32_t>(wave) * 256u));
  };
  constexpr int kPerStage = S::kDmaA + S::kDmaB + (kScaled ? 1 : 0);

  const int frag_row = lane % 16;
  const int frag_kgrp = lane / 16;
  // Pieces frag_piece and frag_piece + 4 of a row: any order does that is the
  // same for both operands.
  const int frag_piece = ((frag_kgrp & 1) << 1) | (frag_kgrp >> 1);
  const uint32_t piece0 = static_cast<uint32_t>((frag_piece ^ S::swz(frag_row)) * 16);
  const uint32_t piece1 = static_cast<uint32_t>(((frag_piece + 4) ^ S::swz(frag_row)) * 16);
  const uint32_t a_base = static_cast<uint32_t>(wm * S::kWaveM + frag_row) * S::kRowBytes;
  const uint32_t b_base = static_cast<uint32_t>(wn * S::kWaveN + frag_row) * S::kRowBytes + S::kStageA;
  const uint32_t sa_base = S::kStageScales + static_cast<uint32_t>(wm * S::kWaveM + frag_row) * 4u;
  const uint32_t sb_base =
      S::kStageScales + static_cast<uint32_t>(S::kScalesA + wn * S::kWaveN + (SB == 1 ? 4 * frag_kgrp : 0)) * 4u;

  int8_v fa[2][S::kFragM], fb[2][S::kFragN];
  float sa[2][S::kFragM];
  float4_t sb[2][S::kFragN];
  float4_t acc[S::kFragM][S::kFragN];
#pragma unroll
  for (int i = 0; i < S::kFragM; ++i)
#pragma unroll
    for (int j = 0; j < S::kFragN; ++j) acc[i][j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  auto read = [&](auto buffer, int slot) {
    constexpr int P = decltype(buffer)::value;
    const char *stage = ring + slot * S::kStageBytes;
    auto block = [&](const char *row) {
      return join(*reinterpret_cast<const int4_t *>(row + piece0), *reinterpret_cast<const int4_t *>(row + piece1));
    };
#pragma unroll
    for (int i = 0; i < S::kFragM; ++i) {
      fa[P][i] = block(stage + a_base + i * 16 * S::kRowBytes);
      if constexpr (kScaled) sa[P][i] = *reinterpret_cast<const float *>(stage + sa_base + i * 64);
    }
#pragma unroll
    for (int j = 0; j < S::kFragN; ++j) {
      fb[P][j] = block(stage + b_base + j * 16 * S::kRowBytes);
      if constexpr (kScaled) {
        if constexpr (SB == 1)
          sb[P][j] = *reinterpret_cast<const float4_t *>(stage + sb_base + j * 64);
        else if (j == 0)
          sb[P][0][0] = *reinterpret_cast<const float *>(stage + sb_base);
      }
    }
  };
  auto products = [&](auto buffer) {
    constexpr int P = decltype(buffer)::value;
#pragma unroll
    for (int j = 0; j < S::kFragN; ++j) {
      if constexpr (kScaled) {
        float4_t part[S::kFragM];
#pragma unroll
        for (int i = 0; i < S::kFragM; ++i) part[i] = mfma_fp8(fb[P][j], fa[P][i], float4_t{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
        for (int i = 0; i < S::kFragM; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][j][e] = __builtin_fmaf(part[i][e], sa[P][i] * sb[P][SB == 1 ? j : 0][SB == 1 ? e : 0], acc[i][j][e]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < S::kFragM; ++i) {
            const int4_t b4 = half_of(fb[P][j], h), a4 = half_of(fa[P][i], h);
            if constexpr (IN == kF16)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, b4),
                                                                 __builtin_bit_cast(half8_t, a4), acc[i][j], 0, 0, 0);
            else
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b4),
                                                                  __builtin_bit_cast(bf16x8_t, a4), acc[i][j], 0, 0, 0);
          }
      }
    }
  };

#pragma unroll
  for (int s = 0; s < S::STAGES; ++s) issue(s, s);
  wait_vmcnt<(S::STAGES - 1) * kPerStage>();
  workgroup_barrier();
  using Even = std::integral_constant<int, 0>;
  using Odd = std::integral_constant<int, 1>;
  read(Even{}, 0);
  int slot = 0;  // of the K tile in registers
  auto step = [&](auto now, auto then, int kt) {
    const int next = slot + 1 == S::STAGES ? 0 : slot + 1;
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    wait_vmcnt<(S::STAGES - 2) * kPerStage>();
    workgroup_barrier();
    __builtin_amdgcn_sched_barrier(0);
    issue(kt + S::STAGES, slot);
    read(then, next);
    products(now);
    __builtin_amdgcn_sched_barrier(0);
    slot = next;
  };
  int kt = 0;
  const int mine = (KT + S::TEAMS - 1) / S::TEAMS;  // K tiles of a team
  for (; kt + 1 < mine; kt += 2) {
    step(Even{}, Odd{}, kt);
    step(Odd{}, Even{}, kt + 1);
  }
  if (kt < mine) products(Even{});

  // The staged output lies over the ring.
  __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  wait_vmcnt<0>();
  workgroup_barrier();
  if constexpr (S::TEAMS > 1) {
    // The teams' sums, joined in their order.
    constexpr int kBlocks = S::kFragM * S::kFragN;
    float4_t *const sums = reinterpret_cast<float4_t *>(smem) + wave * kBlocks * 64 + lane;
    constexpr int kTeam = S::kWaves * kBlocks * 64;
    static_assert((S::TEAMS - 1) * kTeam * 16 + S::kWaves * S::kWaveM * S::kTilePitch <= S::kRingBytes, "LDS");
#pragma unroll
    for (int i = 0; i < S::kFragM; ++i)
#pragma unroll
      for (int j = 0; j < S::kFragN; ++j)
        if (team > 0) sums[(team - 1) * kTeam + (i * S::kFragN + j) * 64] = acc[i][j];
    __syncthreads();
    if (team > 0) return;
#pragma unroll
    for (int t = 0; t < S::TEAMS - 1; ++t)
#pragma unroll
      for (int i = 0; i < S::kFragM; ++i)
#pragma unroll
        for (int j = 0; j < S::kFragN; ++j) acc[i][j] += sums[t * kTeam + (i * S::kFragN + j) * 64];
  }
  char *const tile = smem + (S::TEAMS - 1) * S::kWaves * S::kFragM * S::kFragN * 1024 + wave * S::kWaveM * S::kTilePitch;
#pragma unroll
  for (int i = 0; i < S::kFragM; ++i)
#pragma unroll
    for (int j = 0; j < S::kFragN; ++j) {
      half4_t h;
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = round_out<OUT>(acc[i][j][e]);
      *reinterpret_cast<half4_t *>(tile + (i * 16 + frag_row) * S::kTilePitch + (j * 16 + frag_kgrp * 4) * 2) = h;
    }
  const int n = n0 + wn * S::kWaveN;
  _Float16 *const dst = reinterpret_cast<_Float16 *>(a.D) + (static_cast<int64_t>(m0) + wm * S::kWaveM) * a.N + n;
  store_wave_tile<S::kWaveM, S::kWaveN, S::kTilePitch>(tile, dst, a.N, rows - wm * S::kWaveM, a.N - n, a.alignment, lane);
}

using Deep128x64 = DeepShape<128, 64, 2, 2, 2, 3>;
using Deep64x64 = DeepShape<64, 64, 2, 2, 2, 4>;
using Deep32x64 = DeepShape<32, 64, 2, 2, 2, 6>;
using Deep32x32 = DeepShape<32, 32, 2, 1, 4, 4>;

template <class S, int IN, int OUT, bool GROUPED, int SB>
hipError_t launch_tiles(DeepArgs a, hipStream_t stream) {
  a.tiles_m = static_cast<int>(GROUPED ? unit_bound(a.M, a.E, S::BM) : (a.M + S::BM - 1) / S::BM);
  a.tiles_n = (a.N + S::BN - 1) / S::BN;
  const dim3 grid(static_cast<unsigned>(a.tiles_m * a.tiles_n));
  hipLaunchKernelGGL((deep_kernel<S, IN, OUT, GROUPED, SB>), grid, dim3(S::kThreads), 0, stream, a);
  return hipGetLastError();
}

// Whether there are no more tiles than CUs (of groups: whether there are
// expected to be).
template <class S>
bool fits(int64_t M, int64_t N, int64_t E, int num_cus) {
  const int64_t units = E == 1 ? (M + S::BM - 1) / S::BM : expected_units(M, E, S::BM);
  return units * ((N + S::BN - 1) / S::BN) <= num_cus;
}

// The smallest tile that fits.
template <int IN, int OUT, bool GROUPED, int SB>
hipError_t launch_fitting(const DeepArgs &a, int num_cus, hipStream_t stream) {
  if (fits<Deep32x32>(a.M, a.N, a.E, num_cus)) return launch_tiles<Deep32x32, IN, OUT, GROUPED, SB>(a, stream);
  if (fits<Deep32x64>(a.M, a.N, a.E, num_cus)) return launch_tiles<Deep32x64, IN, OUT, GROUPED, SB>(a, stream);
  if (fits<Deep64x64>(a.M, a.N, a.E, num_cus)) return launch_tiles<Deep64x64, IN, OUT, GROUPED, SB>(a, stream);
  return launch_tiles<Deep128x64, IN, OUT, GROUPED, SB>(a, stream);
}

}  // namespace

bool few_tiles(int64_t M, int64_t N, int64_t E, int num_cus) {
  return fits<Deep128x64>(M, N, E, num_cus);  // the largest: there are no more of it than of any other
}

void few_tiles_plan(int64_t M, int64_t N, int64_t E, int num_cus, int *rows, int *cols) {
  auto is = [&](auto shape) {
    using S = decltype(shape);
    if (!fits<S>(M, N, E, num_cus)) return false;
    *rows = S::BM;
    *cols = S::BN;
    return true;
  };
  is(Deep32x32{}) || is(Deep32x64{}) || is(Deep64x64{}) || is(Deep128x64{});
}

hipError_t launch_deep_fp8(int out, const void *A, const float *sa, const void *B, const float *sb, int sb_rows, void *D,
                           int M, int N, int K, int num_cus, hipStream_t stream) {
  const DeepArgs a{static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(B), sa, sb, nullptr,
                   static_cast<uint16_t *>(D), M, N, 1, K, 0, 0, row_alignment(D, N)};
  if (sb_rows == 1)
    return out == kBF16 ? launch_fitting<kE4m3, kBF16, false, 1>(a, num_cus, stream)
                        : launch_fitting<kE4m3, kF16, false, 1>(a, num_cus, stream);
  return out == kBF16 ? launch_fitting<kE4m3, kBF16, false, kScaleBlock>(a, num_cus, stream)
                      : launch_fitting<kE4m3, kF16, false, kScaleBlock>(a, num_cus, stream);
}

hipError_t launch_deep_grouped(int dtype, const void *X, const void *W, const int *offsets, void *D, int T, int N, int K,
                               int E, int num_cus, hipStream_t stream) {
  const DeepArgs a{static_cast<const uint8_t *>(X), static_cast<const uint8_t *>(W), nullptr, nullptr, offsets,
                   static_cast<uint16_t *>(D), T, N, E, 2 * K, 0, 0, row_alignment(D, N)};
  return dtype == kBF16 ? launch_fitting<kBF16, kBF16, true, kScaleBlock>(a, num_cus, stream)
                        : launch_fitting<kF16, kF16, true, kScaleBlock>(a, num_cus, stream);
}

hipError_t launch_deep_grouped_fp8(int out, const void *X, const float *sx, const void *W, const float *sw,
                                   const int *offsets, void *D, int T, int N, int K, int E, int num_cus,
                                   hipStream_t stream) {
  const DeepArgs a{static_cast<const uint8_t *>(X), static_cast<const uint8_t *>(W), sx, sw, offsets,
                   static_cast<uint16_t *>(D), T, N, E, K, 0, 0, row_alignment(D, N)};
  return out == kBF16 ? launch_fitting<kE4m3, kBF16, true, kScaleBlock>(a, num_cus, stream)
                      : launch_fitting<kE4m3, kF16, true, kScaleBlock>(a, num_cus, stream);
}

}  // namespace gt
