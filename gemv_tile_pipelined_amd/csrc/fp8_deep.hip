// fp8_deep.hip -- dense products of block-scaled e4m3 operands (fp8_gemm.hip)
// with fewer tiles than CUs.
//
// Such a product is bound by latency: a CU has one tile and walks its K tiles
// one after another (32 of 128x128 outputs took 0.5 us each, whatever M).  So
// tiles are small here, the smallest of which there are no more than CUs, and
// the waves form TEAMS teams that take K tiles in turn, each with a ring of its
// own; together the rings fill the LDS.  A step has one barrier: behind it, all
// waves have the team's K tile kt in registers (its stage is refilled) and kt +
// 1 has landed, whose operands are read while kt's products are formed.  The
// teams' sums are joined in LDS, in order.
//
// Measured (MI355X, us; rows x 4096 x 4096; one column per kernel):
//             streamed  32x32  32x64  64x64  tiles of fp8_gemm.hip
//   M =   4        5.4    6.3    8.3    9.5   15.9
//        17        6.6    6.2    8.2    9.7   16.0
//        64       12.5    7.1    8.6   11.1   16.3
//       128               11.8    9.0   11.0   19.0
//       256               21.5   15.9   11.3   19.0
//       512 (128x64: 17.7)                     19.4
// One team (64x64, 8 stages) 13.8 us at M = 128, four of half the depth 13.2, two
// 11.1; loads issued before a step's reads and MFMAs 11.1, between them 11.6.
// Streaming (stream.hip) reads x again for every 16 rows of W: M = 16 of
// 4096x14336 16.3 and here 12.6, of 28672x4096 30.8 and 27.5; M = 4 11.9 and
// 12.3, 23.8 and 26.8; M = 8 13.3 and 12.3, 27.9 and 28.3.
#include "fp8_common.hpp"
#include "kernels.hpp"
#include "tile_order.hpp"
#include "tile_store.hpp"

#include <type_traits>

namespace gt {

namespace {

struct DeepArgs {
  const uint8_t *A, *B;
  const float *sa, *sb;
  uint16_t *D;
  int M, N, K;
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

template <class S, int OUT, int SB>
__global__ void __launch_bounds__(S::kThreads) fp8_deep_kernel(DeepArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[S::kRingBytes];
  const int lane = threadIdx.x & 63;
  const int team = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) / S::kWaves);
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % S::kWaves);
  const int wm = wave / S::WAVES_N;
  const int wn = wave % S::WAVES_N;
  char *const ring = smem + team * (S::STAGES * S::kStageBytes);
  const uint32_t lds0 = lds_addr(smem) + static_cast<uint32_t>(team) * (S::STAGES * S::kStageBytes);
  const int KT = (a.K + kScaleBlock - 1) / kScaleBlock;

  const TileCoord tc = tile_of(xcd_logical_id(blockIdx.x, gridDim.x), a.tiles_m, a.tiles_n, kGemmGroupM);
  const int m0 = static_cast<int>(tc.tm) * S::BM, n0 = static_cast<int>(tc.tn) * S::BN;
  const int rows = min(S::BM, a.M - m0), cols = min(S::BN, a.N - n0);
  const int4_t rsrc_a = make_buffer_rsrc(a.A + static_cast<int64_t>(m0) * a.K, static_cast<uint32_t>(rows) * a.K);
  const int4_t rsrc_b = make_buffer_rsrc(a.B + static_cast<int64_t>(n0) * a.K, static_cast<uint32_t>(cols) * a.K);
  const int4_t rsrc_sa = make_buffer_rsrc(a.sa + static_cast<int64_t>(m0) * KT, static_cast<uint32_t>(rows) * KT * 4u);
  const int sb_rows = SB == 1 ? cols : (cols + kScaleBlock - 1) / kScaleBlock;
  const int4_t rsrc_sb = make_buffer_rsrc(a.sb + static_cast<int64_t>(n0 / SB) * KT, static_cast<uint32_t>(sb_rows) * KT * 4u);

  const int ld_row = wave * 8 + lane / 8;
  const int ld_k = ((lane % 8) ^ S::swz(ld_row)) * 16;
  const uint32_t ld_off = static_cast<uint32_t>(ld_row) * static_cast<uint32_t>(a.K) + static_cast<uint32_t>(ld_k);
  const uint32_t ld_step = static_cast<uint32_t>(S::kRowStep) * static_cast<uint32_t>(a.K);
  // Scales: wave w loads those of 64 of A's rows followed by B's; waves that
  // have none left load the first ones again, to a place that nothing reads.
  const int scale_part = wave % S::kScaleWaves;
  const bool scale_a = scale_part < S::kScalesA / 64;
  const int scale_row = (scale_a ? scale_part : scale_part - S::kScalesA / 64) * 64 + lane;
  const uint32_t scale_off =
      static_cast<uint32_t>(scale_a || SB == 1 ? scale_row : scale_row / kScaleBlock) * static_cast<uint32_t>(KT) * 4u;
  const int4_t rsrc_s = scale_a ? rsrc_sa : rsrc_sb;
  // K tiles past the last: operands out of range, i.e. zeros, and scales of
  // another row or out of range, which belong to sums that nothing uses.
  // kt: the team's own count.
  auto issue = [&](int own, int slot) {
    const int kt = own * S::TEAMS + team;
    const uint32_t stage = lds0 + static_cast<uint32_t>(slot) * S::kStageBytes;
    const int k0 = kt * kScaleBlock;
    const uint32_t off = k0 + ld_k < a.K ? ld_off + static_cast<uint32_t>(k0) : kOobOffset;
#pragma unroll
    for (int d = 0; d < S::kDmaA + S::kDmaB; ++d) {
      const bool is_a = d < S::kDmaA;
      const int i = is_a ? d : d - S::kDmaA;
      lds_dma_b128(is_a ? rsrc_a : rsrc_b, off + i * ld_step,
                   __builtin_amdgcn_readfirstlane(stage + (is_a ? 0 : S::kStageA) + (i * S::kWaves + wave) * 1024));
    }
    lds_dma_b32(rsrc_s, kt < KT ? scale_off + static_cast<uint32_t>(kt) * 4u : kOobOffset,
                __builtin_amdgcn_readfirstlane(stage + S::kStageScales + static_cast<uint32_t>(wave) * 256u));
  };

  const int frag_row = lane % 16;
  const int frag_kgrp = lane / 16;
  const int frag_piece = ((frag_kgrp & 1) << 1) | (frag_kgrp >> 1);  // and frag_piece + 4
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
      sa[P][i] = *reinterpret_cast<const float *>(stage + sa_base + i * 64);
    }
#pragma unroll
    for (int j = 0; j < S::kFragN; ++j) {
      fb[P][j] = block(stage + b_base + j * 16 * S::kRowBytes);
      if constexpr (SB == 1)
        sb[P][j] = *reinterpret_cast<const float4_t *>(stage + sb_base + j * 64);
      else if (j == 0)
        sb[P][0][0] = *reinterpret_cast<const float *>(stage + sb_base);
    }
  };
  auto products = [&](auto buffer) {
    constexpr int P = decltype(buffer)::value;
#pragma unroll
    for (int j = 0; j < S::kFragN; ++j) {
      float4_t part[S::kFragM];
#pragma unroll
      for (int i = 0; i < S::kFragM; ++i) part[i] = mfma_fp8(fb[P][j], fa[P][i], float4_t{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
      for (int i = 0; i < S::kFragM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][j][e] = __builtin_fmaf(part[i][e], sa[P][i] * sb[P][SB == 1 ? j : 0][SB == 1 ? e : 0], acc[i][j][e]);
    }
  };

#pragma unroll
  for (int s = 0; s < S::STAGES; ++s) issue(s, s);
  wait_vmcnt<(S::STAGES - 1) * S::kPerStage>();
  workgroup_barrier();
  using Even = std::integral_constant<int, 0>;
  using Odd = std::integral_constant<int, 1>;
  read(Even{}, 0);
  int slot = 0;  // of the K tile in registers
  auto step = [&](auto now, auto then, int kt) {
    const int next = slot + 1 == S::STAGES ? 0 : slot + 1;
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    wait_vmcnt<(S::STAGES - 2) * S::kPerStage>();
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

template <class S, int OUT, int SB>
hipError_t launch_deep(DeepArgs a, hipStream_t stream) {
  a.tiles_m = (a.M + S::BM - 1) / S::BM;
  a.tiles_n = (a.N + S::BN - 1) / S::BN;
  const dim3 grid(static_cast<unsigned>(a.tiles_m * a.tiles_n));
  hipLaunchKernelGGL((fp8_deep_kernel<S, OUT, SB>), grid, dim3(S::kThreads), 0, stream, a);
  return hipGetLastError();
}

// The smallest tile of which there are no more than CUs.
template <class S>
bool fits(int64_t M, int64_t N, int num_cus) {
  return (M + S::BM - 1) / S::BM * ((N + S::BN - 1) / S::BN) <= num_cus;
}

template <int OUT, int SB>
hipError_t launch_fitting(const DeepArgs &a, int num_cus, hipStream_t stream) {
  if (fits<Deep32x32>(a.M, a.N, num_cus)) return launch_deep<Deep32x32, OUT, SB>(a, stream);
  if (fits<Deep32x64>(a.M, a.N, num_cus)) return launch_deep<Deep32x64, OUT, SB>(a, stream);
  if (fits<Deep64x64>(a.M, a.N, num_cus)) return launch_deep<Deep64x64, OUT, SB>(a, stream);
  return launch_deep<Deep128x64, OUT, SB>(a, stream);
}

}  // namespace

bool fp8_few_tiles(int64_t M, int64_t N, int num_cus) {
  return fits<Deep128x64>(M, N, num_cus);  // the largest: there are no more of it than of any other
}

hipError_t launch_fp8_deep(int out, const void *A, const float *sa, const void *B, const float *sb, int sb_rows, void *D,
                           int M, int N, int K, int num_cus, hipStream_t stream) {
  const DeepArgs a{static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(B), sa, sb, static_cast<uint16_t *>(D),
                   M, N, K, 0, 0, row_alignment(D, N)};
  if (sb_rows == 1)
    return out == kBF16 ? launch_fitting<kBF16, 1>(a, num_cus, stream) : launch_fitting<kF16, 1>(a, num_cus, stream);
  return out == kBF16 ? launch_fitting<kBF16, kScaleBlock>(a, num_cus, stream) : launch_fitting<kF16, kScaleBlock>(a, num_cus, stream);
}

}  // namespace gt
