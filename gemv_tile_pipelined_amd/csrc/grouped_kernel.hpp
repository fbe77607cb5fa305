// grouped_kernel.hpp -- the tiled products grouped by expert, in 16 bits:
//
//   forward  D[t, n]   = sum_k X[t, k] W[e, n, k]
//   dgrad    dX[t, k]  = sum_n dY[t, n] W[e, n, k]
//   wgrad    dW[e, n, k] = sum_t dY[t, n] X[t, k]     over the rows t of group e
//
// Each is a product "rows x columns" contracted over a third index, run on the
// tile shapes, LDS ring and MFMA schedule of the tiled GEMM (gemm_kernel.hpp,
// ring.hpp).  Two things differ.
//
// Which operand is contiguous along what.  An MFMA lane needs 8 consecutive
// contraction indices of one row.  An operand whose memory is contiguous along
// the contraction (X and W forward, dY in dgrad) is held in LDS as rows of 64
// of them, as in the GEMM.  One that is contiguous along its rows instead (W
// in dgrad, both in wgrad) is loaded as it lies, 64 LDS rows (one for each
// contraction index) of BM or BN elements, and transposed on the way to the
// registers by ds_read_b64_tr_b16: of 16 lanes, lane 4j + i points at elements
// 4i .. 4i + 3 of contraction index j, and lane i receives element i of the
// four indices.  Two such reads make an operand register.  32-byte segments
// of an LDS row are permuted within 256 bytes by an XOR with 3 bits of the
// contraction index, chosen so that the 8 segments that any two lane groups
// read together (groups 0 and 1, or 0 and 2) lie in different banks.
//
// Which tiles there are.  Forward and dgrad cut every group's rows into units
// of BM rows; a persistent workgroup keeps a table of the groups in LDS and
// walks (unit, column tile) pairs in the GEMM's grouped order, so that units
// of one group share the group's weights in L2.  In wgrad the groups'
// outputs are all alike and the contraction differs: workgroups are not
// persistent there, so that whichever finishes takes the next tile.
#pragma once

#include "gemm_kernel.hpp"
#include "groups.hpp"
#include "tile_store.hpp"

namespace gt {

enum : int { kGroupForward = 0, kGroupDgrad = 1, kGroupWgrad = 2 };

struct GroupedArgs {
  const uint16_t *A, *B;  // the output's rows come from A, its columns from B
  uint16_t *D;
  const int *offsets;
  int T, N, K, E;
  int tiles_m, tiles_n;  // column tiles; row tiles of a group's output (wgrad)
  int alignment;         // of D's rows
};

template <int BX>
struct TransposedTile {  // 64 LDS rows (contraction) of BX elements
  static constexpr int kRowBytes = BX * 2;
  static constexpr int kChunks = BX / 8;
  static constexpr int kRowsPerDma = 64 / kChunks;
  static_assert(BX == 128 || BX == 256, "LDS rows of 256 or 512 bytes");
  // XOR of a 32-byte segment's number in LDS row r.
  __host__ __device__ static constexpr int swz(int r) { return (r & 3) | ((((r >> 3) ^ (r >> 4)) & 1) << 2); }
};

__device__ inline half4_t lds_read_transposed(uint32_t addr) {
  typedef short short4_v __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(
      half4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<GT_LDS short4_v *>(static_cast<uintptr_t>(addr))));
}

template <class S, int OP>
__global__ void __launch_bounds__(S::kThreads) __attribute__((amdgpu_waves_per_eu(S::kWaves / 4, S::kWaves / 4)))
grouped_gemm_kernel(GroupedArgs a) {
  static_assert(S::MI == 16 && S::BK == 64 && S::STAGES >= 2 && S::SWIZZLE, "the pipelined 16x16x32 loop");
  constexpr bool kTransA = OP == kGroupWgrad;
  constexpr bool kTransB = OP != kGroupForward;
  constexpr bool kTable = OP != kGroupWgrad;
  // The table lies behind the ring in one allocation, so that the ring starts
  // at LDS address 0 and its offsets fit the instructions.
  __shared__ __attribute__((aligned(1024))) char smem[S::kLdsBytes + (kTable ? sizeof(GroupTable) : 0)];
  GroupTable &table = *reinterpret_cast<GroupTable *>(smem + S::kLdsBytes);

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / S::WAVES_N;
  const int wn = wave % S::WAVES_N;
  const uint32_t lds0 = lds_addr(smem);

  // Row strides (elements) of the operands and the output, columns of the
  // output, and the contraction (per group in wgrad).
  const int lda = OP == kGroupForward ? a.K : a.N;
  const int ldb = a.K;
  const int cols = OP == kGroupForward ? a.N : a.K;

  // ---- loader geometry (gemm_kernel.hpp; TransposedTile above) -------------
  static_assert(S::kRowsPerDma * S::kWaves % 16 == 0, "DMA row blocks must keep swz() per-lane");
  const int ld_row = wave * S::kRowsPerDma + lane / S::kChunks;
  const int ld_kcol = ((lane % S::kChunks) ^ S::swz(ld_row)) * 8;
  constexpr int kRowStep = S::kRowsPerDma * S::kWaves;
  constexpr uint32_t kLdsStep = kRowStep * S::kRowBytes;
  static_assert(kLdsStep == S::kWaves * 1024, "one KiB per wave instruction");
  // A transposed operand's instruction i fills LDS rows i * R + r, r the
  // lane's row of R = kRowsPerDma * kWaves; its segments' XOR flips bit 2
  // with some i (flip below), which moves the lane's column by 64 elements.
  auto trans_geometry = [&](auto tile, uint32_t *row, uint32_t *col) {
    using Tt = decltype(tile);
    *row = static_cast<uint32_t>(wave * Tt::kRowsPerDma + lane / Tt::kChunks);
    *col = static_cast<uint32_t>(((lane % Tt::kChunks) ^ (Tt::swz(static_cast<int>(*row)) << 1)) * 8);
  };
  auto flip = [&](auto tile, int i) {
    using Tt = decltype(tile);
    return Tt::swz(i * Tt::kRowsPerDma * S::kWaves) & 4;
  };
  static_assert(TransposedTile<128>::kRowsPerDma * S::kWaves % 8 == 0 &&
                    TransposedTile<256>::kRowsPerDma * S::kWaves % 8 == 0,
                "instruction i changes only bits 3 and up of an LDS row");
  using TileA = TransposedTile<kTransA ? S::BM : 128>;
  using TileB = TransposedTile<kTransB ? S::BN : 128>;
  uint32_t ta_row, ta_col, tb_row, tb_col;
  trans_geometry(TileA{}, &ta_row, &ta_col);
  trans_geometry(TileB{}, &tb_row, &tb_col);

  // ---- operand-read geometry -----------------------------------------------
  const int frag_row = lane % 16;
  const int frag_kgrp = lane / 16;
  const int frag_kchunk = ((frag_kgrp & 1) << 1) | (frag_kgrp >> 1);
  const int frag_swz = S::swz(frag_row);
  const uint32_t a_row_base = static_cast<uint32_t>(wm * S::kWaveM + frag_row) * S::kRowBytes;
  const uint32_t b_row_base = static_cast<uint32_t>(wn * S::kWaveN + frag_row) * S::kRowBytes + S::kStageA;
  // Transposed: lane 4j + i of group g points at contraction index
  // 8 * frag_kchunk + j (and + 4), elements 4i .. 4i + 3 of block 0; block b
  // flips bits 5 .. 7 of the address with b * 32.
  const int t_row = 8 * frag_kchunk + (frag_row >> 2);
  const uint32_t t_swz = static_cast<uint32_t>(TileA::swz(t_row)) << 5;
  const uint32_t t_col = static_cast<uint32_t>(frag_row & 3) * 8;
  const uint32_t ta_base =
      lds0 + static_cast<uint32_t>(t_row * TileA::kRowBytes) + ((static_cast<uint32_t>(wm * S::kWaveM * 2) + t_col) ^ t_swz);
  const uint32_t tb_base = lds0 + S::kStageA + static_cast<uint32_t>(t_row * TileB::kRowBytes) +
                           ((static_cast<uint32_t>(wn * S::kWaveN * 2) + t_col) ^ t_swz);

  // The first barrier of the next tile's K loop also ends this tile's use of
  // the LDS.
  const int64_t stride = gridDim.x;
  int64_t num_tiles, u;
  int units = 0;
  if constexpr (kTable) {
    build_group_table(&table, a.offsets, a.E, a.T, S::BM);
    __syncthreads();
    units = __builtin_amdgcn_readfirstlane(table.upto[a.E - 1]);
    num_tiles = static_cast<int64_t>(units) * a.tiles_n;
    u = xcd_logical_id(blockIdx.x, gridDim.x);
  } else {
    num_tiles = gridDim.x;
    u = xcd_block_id(blockIdx.x, gridDim.x);
  }
  for (; u < num_tiles; u += stride) {
    // This tile's operands, sizes and place in the output.
    const uint16_t *pa, *pb;
    uint16_t *pd;
    int rows, C, n0, m0 = 0;
    if constexpr (kTable) {
      const TileCoord tc = tile_of(u, units, a.tiles_n, kGemmGroupM);
      const GroupUnit g = table_unit(&table, a.E, S::BM, static_cast<int>(tc.tm));
      n0 = static_cast<int>(tc.tn) * S::BN;
      rows = min(S::BM, g.end - g.row);
      C = OP == kGroupForward ? a.K : a.N;
      pa = a.A + static_cast<int64_t>(g.row) * lda;
      pb = a.B + static_cast<int64_t>(g.group) * a.N * a.K;
      if constexpr (OP == kGroupForward) pb += static_cast<int64_t>(n0) * ldb;
      pd = a.D + static_cast<int64_t>(g.row) * cols;
    } else {
      const int per = a.tiles_m * a.tiles_n;
      const int e = static_cast<int>(u / per);
      const TileCoord tc = tile_of(u - static_cast<int64_t>(e) * per, a.tiles_m, a.tiles_n, kGemmGroupM);
      const GroupRows g = group_rows(__builtin_amdgcn_readfirstlane(a.offsets[e]),
                                     __builtin_amdgcn_readfirstlane(a.offsets[e + 1]), a.T);
      m0 = static_cast<int>(tc.tm) * S::BM;
      n0 = static_cast<int>(tc.tn) * S::BN;
      rows = min(S::BM, a.N - m0);
      C = g.end - g.begin;
      pa = a.A + static_cast<int64_t>(g.begin) * lda;
      pb = a.B + static_cast<int64_t>(g.begin) * ldb;
      pd = a.D + (static_cast<int64_t>(e) * a.N + m0) * cols;
    }
    // A sum over nothing still walks one K tile, all of it out of range: zeros.
    const int KT = max(1, (C + S::BK - 1) / S::BK);

    // Buffer descriptors: of a whole panel where the contraction is
    // contiguous; of K tile kt's rows of it, from column `col0` on, where it
    // is not (rows past the contraction's end read as zeros; columns past the
    // operand's own only reach outputs that are not stored).
    int4_t rsrc_a{}, rsrc_b{};
    if constexpr (!kTransA) rsrc_a = make_buffer_rsrc(pa, static_cast<uint32_t>(rows) * lda * 2u);
    if constexpr (!kTransB) rsrc_b = make_buffer_rsrc(pb, static_cast<uint32_t>(min(S::BN, cols - n0)) * ldb * 2u);
    auto k_rows_rsrc = [&](const uint16_t *p, int ld, int col0, int kt) {
      const int k0 = kt * S::BK;
      const int have = min(S::BK, C - k0);
      return make_buffer_rsrc(p + static_cast<int64_t>(k0) * ld + col0,
                              have > 0 ? static_cast<uint32_t>(have) * ld * 2u - static_cast<uint32_t>(col0) * 2u : 0u);
    };

    // Re-materialised inside the tile loop, as in gemm_kernel: this lane's
    // byte offset in each operand, and the bytes from one load instruction's
    // rows to the next's.
    uint32_t off_a = kTransA ? (ta_row * lda + ta_col) * 2u
                             : static_cast<uint32_t>(ld_row) * lda * 2u + static_cast<uint32_t>(ld_kcol) * 2u;
    uint32_t step_a = static_cast<uint32_t>(kTransA ? TileA::kRowsPerDma * S::kWaves : kRowStep) * lda * 2u;
    int kcol = ld_kcol;
    asm volatile("" : "+v"(off_a), "+v"(kcol), "+s"(step_a));
    uint32_t off_b = off_a, step_b = step_a;  // alike where the operands are
    if constexpr (OP != kGroupForward) {
      off_b = (tb_row * ldb + tb_col) * 2u;
      step_b = static_cast<uint32_t>(TileB::kRowsPerDma * S::kWaves) * ldb * 2u;
      asm volatile("" : "+v"(off_b), "+s"(step_b));
    }

    struct DmaArgs {
      int4_t rsrc;
      uint32_t voffset;
    };
    // Load d of a K tile: descriptors ra and rb, and the K tile's first
    // contraction index (its byte offset and the range test of operands that
    // are contiguous along it).
    auto dma_args = [&](int4_t ra, int4_t rb, int k0, int d) -> DmaArgs {
      const bool is_a = d < S::kDmaA;
      const int i = is_a ? d : d - S::kDmaA;
      const uint32_t step = static_cast<uint32_t>(i) * (is_a ? step_a : step_b);
      if (is_a ? kTransA : kTransB) {
        // The flipped column: bit 6 of the element index, i.e. bit 7 of the
        // byte offset within the row.
        uint32_t off = is_a ? off_a : off_b;
        if (is_a ? flip(TileA{}, i) : flip(TileB{}, i)) {
          const uint32_t col = is_a ? ta_col : tb_col;
          off += ((col ^ 64u) - col) * 2u;
        }
        return DmaArgs{is_a ? ra : rb, off + step};
      }
      const uint32_t off = k0 + kcol < C ? (is_a ? off_a : off_b) + static_cast<uint32_t>(k0) * 2u : kOobOffset;
      return DmaArgs{is_a ? ra : rb, off + step};
    };
    auto lds_of = [&](int kt, int d) {
      const uint32_t at = lds0 + static_cast<uint32_t>((kt % S::STAGES) * S::kStageBytes) +
                          static_cast<uint32_t>(wave) * 1024u +
                          (d < S::kDmaA ? d * kLdsStep : S::kStageA + (d - S::kDmaA) * kLdsStep);
      return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(at));
    };
    auto load_one = [&](int kt, int d) {
      int4_t ra = rsrc_a, rb = rsrc_b;
      if (d < S::kDmaA) {
        if constexpr (kTransA) ra = k_rows_rsrc(pa, lda, m0, kt);
      } else {
        if constexpr (kTransB) rb = k_rows_rsrc(pb, ldb, n0, kt);
      }
      const DmaArgs g = dma_args(ra, rb, kt * S::BK, d);
      lds_dma_b128(g.rsrc, g.voffset, lds_of(kt, d));
    };

    half8_t fa[2][S::kFragM], fb[2][S::kFragN];
    // Operand block `blk` of K step ks from the stage of K tile kt.
    auto read_block = [&](bool is_a, int blk, int kt, int ks) -> half8_t {
      const uint32_t stage = static_cast<uint32_t>((kt % S::STAGES) * S::kStageBytes);
      if (is_a ? kTransA : kTransB) {
        const uint32_t rb = is_a ? TileA::kRowBytes : TileB::kRowBytes;
        const uint32_t at =
            ((is_a ? ta_base : tb_base) ^ (static_cast<uint32_t>(blk) << 5)) + stage + static_cast<uint32_t>(ks) * 32u * rb;
        const half4_t lo = lds_read_transposed(at), hi = lds_read_transposed(at + 4 * rb);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
      const uint32_t chunk = static_cast<uint32_t>(((ks * 4 + frag_kchunk) ^ frag_swz) * 16);
      return *reinterpret_cast<const half8_t *>(smem + stage + (is_a ? a_row_base : b_row_base) +
                                                blk * 16 * S::kRowBytes + chunk);
    };
    auto read_frag = [&](int buf, int kt, int ks, int r) {
      if (r == 0)
        fa[buf][0] = read_block(true, 0, kt, ks);
      else if (r <= S::kFragN)
        fb[buf][r - 1] = read_block(false, r - 1, kt, ks);
      else
        fa[buf][r - S::kFragN] = read_block(true, r - S::kFragN, kt, ks);
    };

    float4_t acc[S::kFragM][S::kFragN];
    auto init_acc = [&]() {
#pragma unroll
      for (int i = 0; i < S::kFragM; ++i)
#pragma unroll
        for (int j = 0; j < S::kFragN; ++j) acc[i][j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      // The zeros precede every hand-written MFMA by its wait states
      // (gemm_kernel's accumulator fence).
      static_assert(S::kFragN % 4 == 0, "accumulator fence covers 4 blocks per statement");
#pragma unroll
      for (int i = 0; i < S::kFragM; ++i)
#pragma unroll
        for (int j = 0; j < S::kFragN; j += 4)
          asm volatile("s_nop 1" : "+a"(acc[i][j]), "+a"(acc[i][j + 1]), "+a"(acc[i][j + 2]), "+a"(acc[i][j + 3]));
    };
    auto mfma = [&](int buf, int idx) {
      const int i = S::mfma_i(idx);
      const int j = S::mfma_j(idx);
      if constexpr (S::DTYPE == kF16)
        asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc[i][j]) : "v"(fb[buf][j]), "v"(fa[buf][i]));
      else
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc[i][j]) : "v"(fb[buf][j]), "v"(fa[buf][i]));
    };

    // The refill's descriptors, offsets and LDS address, worked out ahead of
    // the loads that the early-free schedule pairs with MFMAs.
    int4_t rf_a{}, rf_b{};
    uint32_t rf_lds = 0;
    int rf_k0 = 0;
    auto prep = [&](int tile, int part) {
      if (part == 0) {
        rf_k0 = tile * S::BK;
        asm volatile("" : "+s"(rf_k0));
      } else if (part == 1) {
        rf_lds = lds_of(tile, 0);
        asm volatile("" : "+s"(rf_lds));
      } else if (part == 2) {
        rf_a = rsrc_a;
        if constexpr (kTransA) rf_a = k_rows_rsrc(pa, lda, m0, tile);
      } else if (part == 3) {
        rf_b = rsrc_b;
        if constexpr (kTransB) rf_b = k_rows_rsrc(pb, ldb, n0, tile);
      }
    };
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    auto mfma_load = [&](int buf, int idx, int tile, int d) {
      const int i = S::mfma_i(idx);
      const int j = S::mfma_j(idx);
      (void)tile;
      const DmaArgs g = dma_args(rf_a, rf_b, rf_k0, d);
      const uint32_t lds = rf_lds + (d < S::kDmaA ? d * kLdsStep : S::kStageA + (d - S::kDmaA) * kLdsStep);
      if constexpr (S::DTYPE == kF16)
        asm volatile(
            "s_mov_b32 m0, %3\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
            : "+a"(acc[i][j])
            : "v"(fb[buf][j]), "v"(fa[buf][i]), "s"(lds), "v"(g.voffset), "s"(g.rsrc)
            : "memory", "m0");
      else
        asm volatile(
            "s_mov_b32 m0, %3\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
            : "+a"(acc[i][j])
            : "v"(fb[buf][j]), "v"(fa[buf][i]), "s"(lds), "v"(g.voffset), "s"(g.rsrc)
            : "memory", "m0");
    };
#pragma clang diagnostic pop
    KernelRingOps<S, decltype(mfma), decltype(read_frag), decltype(load_one), decltype(mfma_load), decltype(prep),
                  decltype(init_acc)>
        ops{mfma, read_frag, load_one, mfma_load, prep, init_acc};
    if constexpr (S::EARLY_FREE)
      ring_k_loop_ef<S>(ops, KT);
    else
      ring_k_loop<S>(ops, KT);

    // ---- epilogue: as gemm_kernel's, in units' rows ------------------------
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    workgroup_barrier();  // every wave is done reading the ring
    // The lane, made new for every tile: the epilogue's addresses would
    // otherwise be worked out ahead of the tile loop and spilled.
    int ep_lane = lane;
    asm volatile("" : "+v"(ep_lane));
    const int ep_row = ep_lane % 16;
    const int ep_kgrp = ep_lane / 16;
    char *const tile = smem + wave * S::kWaveM * S::kStagePitch;
    const int n = n0 + wn * S::kWaveN;
    _Float16 *const dst = reinterpret_cast<_Float16 *>(pd) + static_cast<int64_t>(wm * S::kWaveM) * cols + n;
#pragma unroll
    for (int i = 0; i < S::kFragM; ++i) {
      const int r = i * 16 + ep_row;
#pragma unroll
      for (int j = 0; j < S::kFragN; ++j) {
        half4_t h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = round_out<S::DTYPE>(acc[i][j][e]);
        *reinterpret_cast<half4_t *>(tile + r * S::kStagePitch + (j * 16 + ep_kgrp * 4) * 2) = h;
      }
      __builtin_amdgcn_sched_barrier(0);  // a block row at a time, for the registers
    }
    store_wave_tile<S::kWaveM, S::kWaveN, S::kStagePitch>(tile, dst, cols, rows - wm * S::kWaveM, cols - n, a.alignment,
                                                          ep_lane);
  }
}

// Expected units of `rows` rows for T rows in E groups whose sizes are not
// known on the host: T / rows whole ones, and half a unit more for each group
// that can have rows.
inline int64_t expected_units(int64_t T, int64_t E, int64_t rows) {
  const int64_t some = E < T ? E : T;
  const int64_t units = T / rows + (some + 1) / 2;
  const int64_t bound = unit_bound(T, E, rows);
  return units < bound ? units : bound;
}

// The tile with the least estimated time (gemm_default_tile's estimate, with
// the units expected instead of row tiles).
inline GemmTile grouped_default_tile(int op, int64_t T, int64_t N, int64_t K, int64_t E, int num_cus) {
  int best = kTile256x256;
  int64_t best_cost = -1;
  for (int t = 0; t <= kTile128x128; ++t) {
    const GemmTileShape &s = kGemmTileShapes[t];
    const int64_t cols = op == kGroupForward ? N : K;
    const int64_t down = op == kGroupWgrad ? E * ((N + s.bm - 1) / s.bm) : expected_units(T, E, s.bm);
    const int64_t tiles = down * ((cols + s.bn - 1) / s.bn);
    const int64_t cost = (tiles + num_cus - 1) / num_cus * s.bm * s.bn * 100 / s.rate_pct;
    if (best_cost < 0 || cost < best_cost) {
      best = t;
      best_cost = cost;
    }
  }
  return static_cast<GemmTile>(best);
}

template <class S, int OP>
static hipError_t launch_grouped_shape(GroupedArgs a, int num_cus, hipStream_t stream) {
  const int cols = OP == kGroupForward ? a.N : a.K;
  a.tiles_n = (cols + S::BN - 1) / S::BN;
  a.tiles_m = (a.N + S::BM - 1) / S::BM;
  a.alignment = row_alignment(a.D, cols);
  int64_t grid;
  if constexpr (OP == kGroupWgrad) {
    grid = static_cast<int64_t>(a.E) * a.tiles_m * a.tiles_n;
  } else {
    const int64_t tiles = unit_bound(a.T, a.E, S::BM) * a.tiles_n;
    grid = tiles < num_cus ? tiles : num_cus;
  }
  hipLaunchKernelGGL((grouped_gemm_kernel<S, OP>), dim3(static_cast<unsigned>(grid)), dim3(S::kThreads), 0, stream, a);
  return hipGetLastError();
}

template <int DT, int OP>
static hipError_t launch_grouped_op(const void *A, const void *B, const int *offsets, void *D, int T, int N, int K, int E,
                                    int num_cus, hipStream_t stream) {
  using Big = std::conditional_t<DT == kF16, GemmDefault, GemmBf16>;
  const GroupedArgs a{static_cast<const uint16_t *>(A), static_cast<const uint16_t *>(B), static_cast<uint16_t *>(D),
                      offsets, T, N, K, E, 0, 0, 0};
  switch (grouped_default_tile(OP, T, N, K, E, num_cus)) {
    case kTile256x128:
      return launch_grouped_shape<GemmTile256x128<DT, kGemmTileShapes[kTile256x128].stages>, OP>(a, num_cus, stream);
    case kTile128x256:
      return launch_grouped_shape<GemmTile128x256<DT, kGemmTileShapes[kTile128x256].stages>, OP>(a, num_cus, stream);
    case kTile128x128:
      return launch_grouped_shape<GemmTile128x128<DT, kGemmTileShapes[kTile128x128].stages>, OP>(a, num_cus, stream);
    default:
      return launch_grouped_shape<Big, OP>(a, num_cus, stream);
  }
}

}  // namespace gt
