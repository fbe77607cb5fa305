// fp8_gemm.hip -- tiled products of block-scaled e4m3 operands, dense and
// grouped:
//
//   D[m, n] = sum_b sa[m, b] sb[n / r, b] sum_{k in block b} A[m, k] B[n, k]
//
// A K tile is one scale block of 128 columns, i.e. 128-byte LDS rows and one
// 16x16x128 MFMA per 16x16 outputs, whose sum is scaled and added to an FP32
// accumulator by four FMAs: the scales change from block to block, so the
// matrix cores cannot accumulate across blocks themselves.  The FMAs need the
// accumulators in ordinary VGPRs (not AGPRs), 256 of which a wave has beside
// nothing else if two waves share a SIMD; hence 8 waves with 64x128 outputs
// each (128 accumulators) on a 256x256 tile, two to a SIMD.  One wave's FMAs and
// LDS reads were to run beside the other's MFMAs, but the counters show little
// of that: MFMAs take 63 % of a SIMD's cycles at 4096^3 and vector instructions
// 38 %, one after the other.
//
// The ring holds STAGES K tiles: the operands' rows (direct-to-LDS loads,
// swizzled as in gemm_kernel.hpp) and the scale of every row of A and of B for
// this block (one 4-byte direct-to-LDS load per wave; with r = 128 rows of B
// that share a scale load it again).  Operand order and epilogue are the
// GEMM's: B first, so that a lane holds 4 consecutive columns of one row, its
// row's scale is one number per 16 rows, and rows leave through LDS as whole
// lines.  With 256x256 tiles and 16-byte aligned rows the next tile's first
// loads go out before this one's stores (8192x8192x1024 81.5 -> 76.6 us), staged
// behind the ring; 128x128 tiles keep the LDS that this takes for a second
// workgroup on the CU (2048 rows over 8 groups x 2048 x 2048: 19.4 us, 29 with
// loads ahead).
//
// Bound by MFMAs and vector instructions in sum, and by the power they draw:
// 4096^3 58 to 61 us, 2.3 PFLOP/s, 8192^3 434 us, 2.5 PFLOP/s.  With a scale for
// each row of B (r = 1) every FMA needs a product of scales beside it, eight VALU
// instructions for each MFMA: 4000x4096x4112 76 us (with 4035 odd columns 85;
// there MFMAs take 38 % of the cycles and vector instructions 45 %).
#include "fp8_common.hpp"
#include "groups.hpp"
#include "kernels.hpp"
#include "tile_store.hpp"

#include <type_traits>

namespace gt {

namespace {

typedef uint32_t uint4_v __attribute__((ext_vector_type(4)));
constexpr int kStreamedStore = 2;  // cache policy: nt

struct Fp8Args {
  const uint8_t *A, *B;
  const float *sa, *sb;
  const int *offsets;
  uint16_t *D;
  int M, N, K, E;  // M: rows of A (all groups)
  int tiles_n;
  int alignment;  // of D's rows
};

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_>
struct Fp8Shape {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, STAGES = STAGES_;
  static constexpr int kWaves = WAVES_M * WAVES_N;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kWaveM = BM / WAVES_M, kWaveN = BN / WAVES_N;
  static constexpr int kFragM = kWaveM / 16, kFragN = kWaveN / 16;
  static constexpr int kRowBytes = kScaleBlock;
  static constexpr int kRowsPerDma = 1024 / kRowBytes;
  static constexpr int kDmaA = BM / kRowsPerDma / kWaves, kDmaB = BN / kRowsPerDma / kWaves;
  static constexpr int kStageA = BM * kRowBytes;
  static constexpr int kStageScales = (BM + BN) * kRowBytes;  // then BM + BN scales
  static constexpr int kStageBytes = kStageScales + (BM + BN) * 4;
  static constexpr int kPerStage = kDmaA + kDmaB + 1;
  static constexpr int kRingBytes = STAGES * kStageBytes;
  // Staging of the output: blocks of 16 rows x 64 columns per wave behind the
  // ring, or (rows that are not 16-byte aligned) whole tiles over it.
  static constexpr bool kLoadAhead = kWaves == 8;
  static constexpr int kBlockPitch = 64 * 2 + 16;
  static constexpr int kBlockBytes = kWaves * 16 * kBlockPitch;
  static constexpr int kStores = kWaveM * kWaveN / 512;  // per wave and tile, 16 bytes a lane
  static constexpr int kTilePitch = kWaveN * 2 + 16;
  static constexpr int kTileBytes = kWaves * kWaveM * kTilePitch;
  static constexpr int lds_bytes(bool aligned) {
    return aligned ? kRingBytes + kBlockBytes : kRingBytes > kTileBytes ? kRingBytes : kTileBytes;
  }
  static_assert((BM + BN) / 64 == kWaves, "one scale load per wave and stage");
  static_assert(kRowsPerDma * kWaves % 16 == 0 && BM % (kRowsPerDma * kWaves) == 0 && BN % (kRowsPerDma * kWaves) == 0,
                "operand loads");
  static_assert(kScaleBlock % kWaveN == 0, "a wave's columns share a scale of B when r = 128");
  static_assert((STAGES - 1) * kPerStage <= 63, "vmcnt range");
  // As GemmShape::swz for 128-byte rows.
  __host__ __device__ static constexpr int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }
};

template <class S, int OUT, bool GROUPED, int SB, bool ALIGNED>
__global__ void __launch_bounds__(S::kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
fp8_gemm_kernel(Fp8Args a) {
  // The table lies behind the ring in one allocation, so that the ring starts
  // at LDS address 0 and its offsets fit the instructions.
  __shared__ __attribute__((aligned(1024))) char smem[S::lds_bytes(ALIGNED) + (GROUPED ? sizeof(GroupTable<kMaxGroups>) : 0)];
  auto &table = *reinterpret_cast<GroupTable<kMaxGroups> *>(smem + S::lds_bytes(ALIGNED));
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / S::WAVES_N;
  const int wn = wave % S::WAVES_N;
  const uint32_t lds0 = lds_addr(smem);
  const int KT = (a.K + kScaleBlock - 1) / kScaleBlock;

  const int ld_row = wave * S::kRowsPerDma + lane / 8;
  const int ld_k = ((lane % 8) ^ S::swz(ld_row)) * 16;
  constexpr int kRowStep = S::kRowsPerDma * S::kWaves;
  const uint32_t ld_off = static_cast<uint32_t>(ld_row) * static_cast<uint32_t>(a.K) + static_cast<uint32_t>(ld_k);
  const uint32_t ld_step = static_cast<uint32_t>(kRowStep) * static_cast<uint32_t>(a.K);
  // Scales: wave w loads those of rows 64 w .. 64 w + 63 of A's rows followed
  // by B's.
  const bool scale_a = wave < S::BM / 64;
  const int scale_row = (scale_a ? wave : wave - S::BM / 64) * 64 + lane;
  const uint32_t scale_off =
      static_cast<uint32_t>(scale_a || SB == 1 ? scale_row : scale_row / kScaleBlock) * static_cast<uint32_t>(KT) * 4u;

  const int frag_row = lane % 16;
  const int frag_kgrp = lane / 16;
  const int frag_piece = ((frag_kgrp & 1) << 1) | (frag_kgrp >> 1);  // and frag_piece + 4
  const uint32_t piece0 = static_cast<uint32_t>((frag_piece ^ S::swz(frag_row)) * 16);
  const uint32_t piece1 = static_cast<uint32_t>(((frag_piece + 4) ^ S::swz(frag_row)) * 16);
  const uint32_t a_base = static_cast<uint32_t>(wm * S::kWaveM + frag_row) * S::kRowBytes;
  const uint32_t b_base = static_cast<uint32_t>(wn * S::kWaveN + frag_row) * S::kRowBytes + S::kStageA;
  const uint32_t sa_base = S::kStageScales + static_cast<uint32_t>(wm * S::kWaveM + frag_row) * 4u;
  const uint32_t sb_base =
      S::kStageScales + static_cast<uint32_t>(S::BM + wn * S::kWaveN + (SB == 1 ? 4 * frag_kgrp : 0)) * 4u;

  int units = (a.M + S::BM - 1) / S::BM;
  if constexpr (GROUPED) {
    build_group_table(&table, a.offsets, a.E, a.M, S::BM);
    __syncthreads();
    units = table_units(&table, a.E);
  }
  const int64_t num_tiles = static_cast<int64_t>(units) * a.tiles_n;
  // A tile's descriptors, sizes and place in the output.
  struct Tile {
    int4_t rsrc_a, rsrc_b, rsrc_s;  // this wave's rows of scales
    int row, rows, n0;
  };
  auto locate = [&](int64_t u) -> Tile {
    GroupUnit g{0, 0, a.M};
    int tn;
    if constexpr (GROUPED) {
      g = table_tile(&table, a.E, S::BM, a.tiles_n, u, &tn);
    } else {
      const TileCoord tc = tile_of(u, units, a.tiles_n, kGemmGroupM);
      g.row = static_cast<int>(tc.tm) * S::BM;
      tn = static_cast<int>(tc.tn);
    }
    Tile t;
    t.n0 = tn * S::BN;
    t.row = g.row;
    t.rows = min(S::BM, g.end - g.row);
    const int cols = min(S::BN, a.N - t.n0);
    const int64_t b_row = static_cast<int64_t>(g.group) * a.N + t.n0;
    t.rsrc_a = make_buffer_rsrc(a.A + static_cast<int64_t>(g.row) * a.K, static_cast<uint32_t>(t.rows) * a.K);
    t.rsrc_b = make_buffer_rsrc(a.B + b_row * a.K, static_cast<uint32_t>(cols) * a.K);
    const int64_t sb_row =
        SB == 1 ? b_row
                : static_cast<int64_t>(g.group) * ((a.N + kScaleBlock - 1) / kScaleBlock) + t.n0 / kScaleBlock;
    const int sb_rows = SB == 1 ? cols : (cols + kScaleBlock - 1) / kScaleBlock;
    t.rsrc_s = make_buffer_rsrc((scale_a ? a.sa + static_cast<int64_t>(g.row) * KT : a.sb + sb_row * KT),
                                static_cast<uint32_t>(scale_a ? t.rows : sb_rows) * KT * 4u);
    return t;
  };
  uint32_t tile_off;
  int tile_k;
  auto lane_offsets = [&]() {
    tile_off = ld_off;
    tile_k = ld_k;
    asm volatile("" : "+v"(tile_off), "+v"(tile_k));
  };
  // Load d of this wave for K tile kt (A's rows, B's rows, then the scales).
  auto issue_one = [&](const Tile &t, int kt, int d) {
    const uint32_t stage = lds0 + static_cast<uint32_t>((kt % S::STAGES) * S::kStageBytes);
    const int k0 = kt * kScaleBlock;
    if (d < S::kDmaA + S::kDmaB) {
      const bool is_a = d < S::kDmaA;
      const int i = is_a ? d : d - S::kDmaA;
      const uint32_t off = k0 + tile_k < a.K ? tile_off + static_cast<uint32_t>(k0) : kOobOffset;
      lds_dma_b128(is_a ? t.rsrc_a : t.rsrc_b, off + i * ld_step,
                   __builtin_amdgcn_readfirstlane(stage + (is_a ? 0 : S::kStageA) + (i * S::kWaves + wave) * 1024));
    } else {
      lds_dma_b32(t.rsrc_s, scale_off + static_cast<uint32_t>(kt) * 4u,
                  __builtin_amdgcn_readfirstlane(stage + S::kStageScales + static_cast<uint32_t>(wave) * 256u));
    }
  };

  // Loads are issued in two parts.  The first half of each wave column's
  // blocks of B lies in the even loads of B's rows, the second in the odd.
  constexpr int kEarly = S::kDmaA + S::kDmaB / 2;  // A and B's first half
  constexpr int kLate = S::kPerStage - kEarly;     // the scales, then B's second half
  auto issue_early = [&](const Tile &t, int kt, int k) {
    issue_one(t, kt, k < S::kDmaA ? k : S::kDmaA + 2 * (k - S::kDmaA));
  };
  auto issue_late = [&](const Tile &t, int kt, int k) {
    issue_one(t, kt, k == 0 ? S::kDmaA + S::kDmaB : S::kDmaA + 2 * (k - 1) + 1);
  };
  static_assert(S::kDmaB % 2 == 0 && kRowStep * 2 == S::kWaveN, "a half of a wave column's rows per load of B");
  auto load_ahead = [&](const Tile &t) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int k = 0; k < kEarly; ++k) issue_early(t, s, k);
#pragma unroll
      for (int k = 0; k < kLate; ++k) issue_late(t, s, k);
    }
  };

  int64_t u = xcd_logical_id(blockIdx.x, gridDim.x);
  if (u >= num_tiles) return;
  Tile cur = locate(u);
  lane_offsets();
  load_ahead(cur);
  bool stores = false;  // of the tile before, younger than the loads ahead
  // Until all loads but the last `count` are complete, those stores aside.
  auto wait_loads = [&](auto count, bool and_stores) {
    constexpr int kCount = decltype(count)::value;
    if (ALIGNED && and_stores)
      wait_vmcnt<kCount + S::kStores>();
    else
      wait_vmcnt<kCount>();
  };
  using Ahead = std::integral_constant<int, kLate - 1 + S::kPerStage>;  // K tile 0 but for B's second half
  using AtFirst = std::integral_constant<int, kEarly + kLate>;           // k_tile's first barrier
  using AtSecond = std::integral_constant<int, kLate - 1 + kEarly>;      // and its second
  for (;;) {
    lane_offsets();
    // A wave whose rows lie behind the last one loads its share, and leaves the
    // matrix units to the wave that shares its SIMD (4 waves on or back, 128
    // rows away): 1000x4096x7168 37.7 -> 36.0 us.
    const bool idle = wm * S::kWaveM >= cur.rows;
    // Operands in registers: all 16-row blocks of A for a K tile, and the
    // current and next block of B; scales of A's rows (times the one of B's
    // columns if they share it) of this K tile and the one before.
    float4_t acc[S::kFragM][S::kFragN], part[S::kFragM], sbv[2];
    int8_v fa[S::kFragM], fb[2];
    float sa[2][S::kFragM];
    auto read_a = [&](const char *stage, int i) {
      const char *row = stage + a_base + i * 16 * S::kRowBytes;
      fa[i] = join(*reinterpret_cast<const int4_t *>(row + piece0), *reinterpret_cast<const int4_t *>(row + piece1));
    };
    auto read_b = [&](const char *stage, int j) {
      const char *row = stage + b_base + j * 16 * S::kRowBytes;
      fb[j & 1] = join(*reinterpret_cast<const int4_t *>(row + piece0), *reinterpret_cast<const int4_t *>(row + piece1));
    };
    auto read_scales = [&](const char *stage, int buf) {
      const float sb = SB == 1 ? 1.0f : *reinterpret_cast<const float *>(stage + sb_base);
#pragma unroll
      for (int i = 0; i < S::kFragM; ++i) {
        sa[buf][i] = *reinterpret_cast<const float *>(stage + sa_base + i * 64);
        if constexpr (SB != 1) sa[buf][i] *= sb;
      }
    };
    // Add the scaled sum of MFMA slot m of a K tile whose scales are in sa[buf].
    auto accumulate = [&](int m, int buf) {
      const int i = m % S::kFragM, j = m / S::kFragM;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[i][j][e] = __builtin_fmaf(part[i][e], SB == 1 ? sa[buf][i] * sbv[j & 1][e] : sa[buf][i], acc[i][j][e]);
      asm volatile("" : "+v"(acc[i][j]));  // here, and not where the sums are used next
    };
    // One K tile, fixed in order: per MFMA slot the MFMA, the four FMAs of the
    // slot three before it (whose MFMA has long finished), and what has to be
    // read or loaded meanwhile.  B's blocks are read one block ahead.  Two
    // barriers let every load fly for about 1.5 K tiles, two stages
    // notwithstanding:
    //  * the first, before the last block of B's first half: all of A (read
    //    during the K tile before) and of B's first half is in registers, so
    //    that part of the stage is refilled; and B's second half has landed;
    //  * the second, before the last block: the rest is in registers and is
    //    refilled, and the next K tile's A, first half of B and scales have
    //    landed, the blocks of A being read into the registers of this one's as
    //    its last MFMA on each is issued.
    // Loads complete in order: what may still be in flight at a barrier is
    // what was issued after what it needs.
    constexpr int kSlots = S::kFragM * S::kFragN;
    constexpr int kBehind = 3;
    constexpr int kFirst = (S::kFragN / 2 - 1) * S::kFragM, kSecond = kSlots - S::kFragM;
    static_assert(S::STAGES == 2 && S::kFragM == 4 && S::kFragN % 2 == 0, "the slots' register reuse");
    static_assert(kFirst + kEarly <= kSecond && kLate <= S::kFragM, "a load per slot");
    auto k_tile = [&](auto parity, auto head, int kt) {
      constexpr int P = decltype(parity)::value;
      constexpr bool kHead = decltype(head)::value;  // K tile 0 or 1
      const char *stage = smem + P * S::kStageBytes;
      const char *other = smem + (1 - P) * S::kStageBytes;
#pragma unroll
      for (int n = 0; n < kSlots; ++n) {
        const int i = n % S::kFragM, j = n / S::kFragM;
        if (n == kFirst || n == kSecond) {
          __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
          // All of K tile kt + 1; or B's second half of kt + 1 and the early
          // part of kt + 2.
          if (n == kFirst)
            wait_loads(AtFirst{}, kHead && stores);
          else
            wait_loads(AtSecond{}, kHead && P == 0 && stores);
          workgroup_barrier();
          __builtin_amdgcn_sched_barrier(0);
        }
        part[i] = mfma_fp8(fb[j & 1], fa[i], float4_t{0.0f, 0.0f, 0.0f, 0.0f});
        __builtin_amdgcn_sched_barrier(0);
        if (n < kBehind)
          accumulate(kSlots - kBehind + n, 1 - P);
        else
          accumulate(n - kBehind, P);
        __builtin_amdgcn_sched_barrier(0);
        // No branches, so that the slots stay in this order: past the last K
        // tile the reads fetch numbers that nothing uses, and the loads, out
        // of range, write zeros that nothing reads.
        if (j + 1 < S::kFragN) {
          if (i == 0) read_b(stage, j + 1);
          if (n >= kFirst && n < kFirst + kEarly) issue_early(cur, kt + 2, n - kFirst);
        } else {
          read_a(other, i);
          if (i == 0) read_b(other, 0);
          if (i == S::kFragM - 1) read_scales(other, 1 - P);
          if (i < kLate) issue_late(cur, kt + 2, i);
        }
        if constexpr (SB == 1) {
          // B's scales of a block, once the slots of the block two before are done.
          if (i == kBehind - 1) sbv[(j + 1) & 1] = *reinterpret_cast<const float4_t *>(
              (j + 1 < S::kFragN ? stage : other) + sb_base + (j + 1) % S::kFragN * 64);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };

#pragma unroll
    for (int i = 0; i < S::kFragM; ++i) {
      part[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      sa[1][i] = 0.0f;  // "before" the first K tile
#pragma unroll
      for (int j = 0; j < S::kFragN; ++j) acc[i][j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    sbv[1] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    wait_loads(Ahead{}, stores);
    workgroup_barrier();
    if (idle) {
      for (int kt = 0; kt < KT; ++kt) {
        wait_loads(AtFirst{}, stores && kt < 2);
        workgroup_barrier();
#pragma unroll
        for (int k = 0; k < kEarly; ++k) issue_early(cur, kt + 2, k);
        wait_loads(AtSecond{}, stores && kt < 1);
        workgroup_barrier();
#pragma unroll
        for (int k = 0; k < kLate; ++k) issue_late(cur, kt + 2, k);
      }
    } else {
#pragma unroll
      for (int i = 0; i < S::kFragM; ++i) read_a(smem, i);
      read_b(smem, 0);
      read_scales(smem, 0);
      if constexpr (SB == 1) sbv[0] = *reinterpret_cast<const float4_t *>(smem + sb_base);
      using Even = std::integral_constant<int, 0>;
      using Odd = std::integral_constant<int, 1>;
      int kt = 0;
      if (ALIGNED && KT > 1) {
        k_tile(Even{}, std::true_type{}, 0);
        k_tile(Odd{}, std::true_type{}, 1);
        kt = 2;
      }
      for (; kt + 1 < KT; kt += 2) {
        k_tile(Even{}, std::false_type{}, kt);
        k_tile(Odd{}, std::false_type{}, kt + 1);
      }
      if (kt < KT) {
        k_tile(Even{}, std::false_type{}, kt);
#pragma unroll
        for (int m = kSlots - kBehind; m < kSlots; ++m) accumulate(m, 0);
      } else {
#pragma unroll
        for (int m = kSlots - kBehind; m < kSlots; ++m) accumulate(m, 1);
      }
    }

    // ---- epilogue ------------------------------------------------------------
    // Every wave has read its last operands before the loop's last barrier: the
    // ring is free, and the next tile's first loads go out ahead of this one's
    // stores (grouped_kernel.hpp).
    const int64_t next_u = u + gridDim.x;
    const bool more = next_u < num_tiles;
    Tile after{};
    if (more) after = locate(next_u);
    if constexpr (ALIGNED) {
      if (more) load_ahead(after);
    }
    // The lane, made new for every tile (grouped_kernel.hpp).
    int ep_lane = lane;
    asm volatile("" : "+v"(ep_lane));
    const int ep_row = ep_lane % 16;
    const int ep_kgrp = ep_lane / 16;
    const int n = cur.n0 + wn * S::kWaveN;
    auto rounded = [&](int i, int j) {
      half4_t h;
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = round_out<OUT>(acc[i][j][e]);
      return h;
    };
    if constexpr (ALIGNED) {
      if (!idle) {
      uint16_t *const pd = a.D + static_cast<int64_t>(cur.row) * a.N;
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
          pd, 0, static_cast<int>(static_cast<uint32_t>(cur.rows) * a.N * 2u), 0x00020000);
      char *const block = smem + S::kRingBytes + wave * 16 * S::kBlockPitch;
      const char *const from = block + ep_lane / 8 * S::kBlockPitch + ep_lane % 8 * 16;
      const int row0 = wm * S::kWaveM + ep_lane / 8;
#pragma unroll
      for (int i = 0; i < S::kFragM; ++i) {
#pragma unroll
        for (int j0 = 0; j0 < S::kFragN; j0 += 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<half4_t *>(block + ep_row * S::kBlockPitch + (j * 16 + ep_kgrp * 4) * 2) =
                rounded(i, j0 + j);
          const int c = n + j0 * 16 + ep_lane % 8 * 8;
#pragma unroll
          for (int r = 0; r < 16; r += 8) {
            const uint4_v v = *reinterpret_cast<const uint4_v *>(from + r * S::kBlockPitch);
            const uint32_t off =
                c < a.N ? static_cast<uint32_t>(row0 + i * 16 + r) * static_cast<uint32_t>(a.N) * 2u +
                              static_cast<uint32_t>(c) * 2u
                        : kOobOffset;
            __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, static_cast<int>(off), 0, kStreamedStore);
          }
        }
      }
      }
      stores = !idle;
    } else {
      wait_vmcnt<0>();  // the loads past the last K tile have written their zeros
      workgroup_barrier();
      char *const tile = smem + wave * S::kWaveM * S::kTilePitch;
#pragma unroll
      for (int i = 0; i < S::kFragM; ++i)
#pragma unroll
        for (int j = 0; j < S::kFragN; ++j)
          *reinterpret_cast<half4_t *>(tile + (i * 16 + ep_row) * S::kTilePitch + (j * 16 + ep_kgrp * 4) * 2) = rounded(i, j);
      _Float16 *const dst =
          reinterpret_cast<_Float16 *>(a.D) + (static_cast<int64_t>(cur.row) + wm * S::kWaveM) * a.N + n;
      store_wave_tile<S::kWaveM, S::kWaveN, S::kTilePitch>(tile, dst, a.N, cur.rows - wm * S::kWaveM, a.N - n,
                                                           a.alignment, ep_lane);
      __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
      workgroup_barrier();  // every wave has read its staged tile
      if (more) load_ahead(after);
    }
    if (!more) break;
    cur = after;
    u = next_u;
  }
}

using Fp8Tile256 = Fp8Shape<256, 256, 4, 2, 2>;
using Fp8Tile128 = Fp8Shape<128, 128, 2, 2, 2>;

template <class S, int OUT, bool GROUPED, int SB>
hipError_t launch_shape(Fp8Args a, int num_cus, hipStream_t stream) {
  a.tiles_n = (a.N + S::BN - 1) / S::BN;
  a.alignment = row_alignment(a.D, a.N);
  const int64_t units = GROUPED ? unit_bound(a.M, a.E, S::BM) : (a.M + S::BM - 1) / S::BM;
  const int64_t tiles = units * a.tiles_n;
  // Workgroups that fit the CUs at once: by LDS, and two waves to a SIMD.
  auto launch = [&](auto aligned) {
    constexpr bool kAligned = decltype(aligned)::value;
    constexpr int kLds = S::lds_bytes(kAligned) + (GROUPED ? static_cast<int>(sizeof(GroupTable<kMaxGroups>)) : 0);
    constexpr int kByLds = 160 * 1024 / kLds, kByWaves = 8 / S::kWaves;
    constexpr int kPerCu = kByLds < kByWaves ? kByLds : kByWaves;
    static_assert(kPerCu >= 1, "a workgroup fits a CU");
    const int64_t fit = static_cast<int64_t>(num_cus) * kPerCu;
    const dim3 grid(static_cast<unsigned>(tiles < fit ? tiles : fit));
    hipLaunchKernelGGL((fp8_gemm_kernel<S, OUT, GROUPED, SB, kAligned>), grid, dim3(S::kThreads), 0, stream, a);
  };
  // A tile's rows have to fit a descriptor's range of the output as well.
  if constexpr (S::kLoadAhead) {
    if (a.alignment == 16 && static_cast<int64_t>(a.N) * S::BM * 2 < (int64_t{1} << 31)) {
      launch(std::true_type{});
      return hipGetLastError();
    }
  }
  launch(std::false_type{});
  return hipGetLastError();
}

// The tile with the shorter estimate: a round of 256x256 tiles, one on each CU,
// takes 1.4 times as long as one of 128x128 tiles, two on each.  Measured (us,
// 128x128 and 256x256): 1024x8192x4096 (one round, one of which half is empty)
// 39 and 49; 1280x8192x4096 (two, one) 72 and 48; 2500x5000x2048 (two, one) 42
// and 38; 4096 rows over 8 groups x 2048 x 2048 (two, one) 37 and 29, over 32
// groups (two, two) 53 and 57.
bool use_tile256(bool grouped, int64_t M, int64_t N, int64_t E, int num_cus) {
  auto tiles = [&](int64_t side) {
    return (grouped ? expected_units(M, E, side) : (M + side - 1) / side) * ((N + side - 1) / side);
  };
  const int64_t big = (tiles(256) + num_cus - 1) / num_cus;
  const int64_t small = (tiles(128) + 2 * num_cus - 1) / (2 * num_cus);
  return 14 * big < 10 * small;
}

template <int OUT, bool GROUPED, int SB>
hipError_t launch_tile(const Fp8Args &a, int num_cus, hipStream_t stream) {
  if (use_tile256(GROUPED, a.M, a.N, a.E, num_cus)) return launch_shape<Fp8Tile256, OUT, GROUPED, SB>(a, num_cus, stream);
  return launch_shape<Fp8Tile128, OUT, GROUPED, SB>(a, num_cus, stream);
}

}  // namespace

hipError_t launch_gemm_fp8(int out, const void *A, const float *sa, const void *B, const float *sb, int sb_rows, void *D,
                           int M, int N, int K, int num_cus, hipStream_t stream) {
  const Fp8Args a{static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(B), sa, sb, nullptr,
                  static_cast<uint16_t *>(D), M, N, K, 1, 0, 0};
  if (sb_rows == 1)
    return out == kBF16 ? launch_tile<kBF16, false, 1>(a, num_cus, stream) : launch_tile<kF16, false, 1>(a, num_cus, stream);
  return out == kBF16 ? launch_tile<kBF16, false, kScaleBlock>(a, num_cus, stream)
                      : launch_tile<kF16, false, kScaleBlock>(a, num_cus, stream);
}

hipError_t launch_grouped_fp8(int out, const void *X, const float *sx, const void *W, const float *sw, const int *offsets,
                              void *D, int T, int N, int K, int E, int num_cus, hipStream_t stream) {
  const Fp8Args a{static_cast<const uint8_t *>(X), static_cast<const uint8_t *>(W), sx, sw, offsets,
                  static_cast<uint16_t *>(D), T, N, K, E, 0, 0};
  return out == kBF16 ? launch_tile<kBF16, true, kScaleBlock>(a, num_cus, stream)
                      : launch_tile<kF16, true, kScaleBlock>(a, num_cus, stream);
}

void fp8_tile(bool grouped, int64_t M, int64_t N, int64_t E, int num_cus, int *rows, int *cols) {
  *rows = *cols = use_tile256(grouped, M, N, E, num_cus) ? 256 : 128;
}

}  // namespace gt
