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
// read together (groups 0 and 1, or 0 and 2) lie in different banks.  Counted, 4 %
// of the LDS cycles of dgrad (one such operand) are conflicts and 20 % of wgrad's
// (both), which that does not account for.
//
// Which tiles there are.  Forward and dgrad cut every group's rows into units
// of BM rows; a persistent workgroup keeps a table of the groups in LDS and
// walks (unit, column tile) pairs group by group (table_tile), so that units
// of one group share the group's weights in L2.  In wgrad the groups' outputs
// are all alike and the contraction differs: the groups' tiles come in order of
// falling length and the workgroups take them forwards and backwards in turn,
// so that each gets about the same sum of lengths.
//
// Between two tiles.  Contractions are short here (a group's rows in wgrad, a
// projection's width), so a tile's start and end count.  The first loads of the
// next tile go out as soon as every wave has read its last operands, before
// this tile's results are rounded and stored.  These pass, a block row at a
// time, through a staging area behind the ring and leave as whole lines by
// buffer stores, always the same number of them, so that the next tile's waits
// can count them.  Outputs whose rows are not 16-byte aligned are staged whole
// over the ring instead (tile_store.hpp), before the next tile's loads.
//
// Bound by the matrix cores, and by tiles that are not full or do not fill the
// last round: 8192 rows in one group x 4096 x 2048 97 to 101 us, 1.4 PFLOP/s, the
// rate of a plain product; over 16 uneven groups (8200 rows in 38 units; 33 would
// hold them, 2.35 rounds) 137 us, dgrad 141; 2.35 rounds at that rate are 114 to
// 119.  Loads ahead, staged stores and one loop body
// took forward from 157 to 142, dgrad from 190 to 145, wgrad from 176 to 161 us.
// Stores straight from the registers, in 64-byte pieces, were slower than staged
// lines.  In wgrad a tile's sum is as short as its group (8 K tiles here), and of
// the 161 us 30 go with the stores (131 us without); giving the XCDs or every
// second workgroup another order of the rounds did not take any of it away, nor
// did other cache policies.
#pragma once

#include "gemm_kernel.hpp"
#include "groups.hpp"
#include "tile_store.hpp"

namespace gt {

typedef uint32_t uint4_v __attribute__((ext_vector_type(4)));
constexpr int kStreamed = 2;  // cache policy of a store: nt

enum : int { kGroupForward = 0, kGroupDgrad = 1, kGroupWgrad = 2 };

struct GroupedArgs {
  const uint16_t *A, *B;  // the output's rows come from A, its columns from B
  uint16_t *D;
  const int *offsets;
  int T, N, K, E;
  int alignment;  // of D's rows
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

// The groups in the order wgrad takes them.
template <int CAP>
struct WgradTable {
  int group[CAP];
  int begin[CAP];
  int end[CAP];
};
// Groups are sorted by length if there are no more than this; among many the
// sums even out by themselves.
constexpr int kMaxSorted = 256;

template <int CAP>
__device__ inline void build_wgrad_table(WgradTable<CAP> *table, const int *__restrict__ offsets, int E, int T, int threads) {
  const int tid = static_cast<int>(threadIdx.x);
  for (int e = tid; e < E; e += threads) {
    const GroupRows g = group_rows(offsets[e], offsets[e + 1], T);
    table->group[e] = e;
    table->begin[e] = g.begin;
    table->end[e] = g.end;
  }
  __syncthreads();
  if (E > kMaxSorted) return;
  const bool mine = tid < E;
  const int begin = mine ? table->begin[tid] : 0, end = mine ? table->end[tid] : 0;
  int rank = 0;
  for (int e = 0; e < E; ++e) {
    const int len = table->end[e] - table->begin[e];
    rank += len > end - begin || (len == end - begin && e < tid);
  }
  __syncthreads();
  if (mine) {
    table->group[rank] = tid;
    table->begin[rank] = begin;
    table->end[rank] = end;
  }
}

// K tiles whose loads are issued ahead of a K loop.
template <class S>
GT_HD constexpr int grouped_ahead() {
  return S::EARLY_FREE ? S::STAGES : S::STAGES - 1;
}

// The vmcnts of the loop's waits: the first, for the oldest K tile of those
// issued ahead, and the one of every K tile after it.
template <class S>
struct GroupedWaits {
  static constexpr int kFirst = (grouped_ahead<S>() - 1) * S::kDmaPerStage;
  static constexpr int loop_count() {
    if constexpr (S::EARLY_FREE)
      return RingEarly<S>::kSteadyVmcnt;
    else
      return (S::STAGES - 2) * S::kDmaPerStage;
  }
  static constexpr int kLoop = loop_count();
  // What a K tile waits for where the walker asks for `n`: never fewer loads
  // than asked for.
  GT_HD static constexpr int in_loop(int n) { return n >= kLoop ? kLoop : 0; }
};

// The ring walker's operations (gemm_kernel.hpp), with waits that let `STORES`
// younger stores of the tile before stay in flight while `stores` is set.
template <class S, int STORES, class Base>
struct GroupedRingOps : Base {
  bool stores;
  __device__ __attribute__((always_inline)) void wait_first(bool and_stores) {
    if (and_stores)
      wait_vmcnt<GroupedWaits<S>::kFirst + STORES>();
    else
      wait_vmcnt<GroupedWaits<S>::kFirst>();
    stores = and_stores;  // the tile that the next wait is for is older than the stores as well
  }
  __device__ __attribute__((always_inline)) void wait_tile(int n) {
    if (GroupedWaits<S>::in_loop(n) != GroupedWaits<S>::kLoop)
      wait_vmcnt<0>();
    else if (stores)
      wait_vmcnt<GroupedWaits<S>::kLoop + STORES>();
    else
      wait_vmcnt<GroupedWaits<S>::kLoop>();
    stores = false;
  }
};

// ring.hpp's K loops from the point where the loads of the first tiles are
// issued, with every K tile in the steady state: loads past the last K tile are
// out of range and write zeros to stages that nothing reads any more, and the
// operands read past it are not used.  The walker is told of STAGES more K
// tiles from each one on, so that its counts are those of the steady state
// however long the sum is.  One loop body instead of one for each phase of the
// ring: through several, the accumulators did not keep their registers.
// `first` is 0 but in the host-side trace.
template <class S, class Ops>
GT_RING_INLINE void grouped_k_loop(Ops &ops, int first, int ktu, bool stores) {
  ops.init_acc();
  ops.fence();
  ops.wait_first(stores);
  ops.barrier();
#pragma unroll
  for (int r = 0; r < S::kReads; ++r) ops.read(0, first, 0, r);
  int kt = first;
  if constexpr (S::EARLY_FREE) {
    for (; kt + 1 < ktu; kt += 2) {
      ring_ktile_ef<S, true, true>(ops, kt, kt + S::STAGES);
      ring_ktile_ef<S, true, true>(ops, kt + 1, kt + 1 + S::STAGES);
    }
    if (kt < ktu) ring_ktile_ef<S, true, true>(ops, kt, kt + S::STAGES);
  } else {
#pragma unroll
    for (int pos = 0; pos < RingSlots<S>::kAfter; ++pos) {
      const int d = ring_slot_load<S>(pos);
      if (d >= 0) ops.load(first + S::STAGES - 1, d);
    }
    for (; kt < ktu; ++kt) ring_ktile<S, true, true, true>(ops, kt, kt + S::STAGES);
  }
}

// Where a tile lies in its group's output (or unit): the operands' rows that
// it is made of, its sizes and its place in the output.
struct GroupedTile {
  const uint16_t *pa, *pb;
  uint16_t *pd;
  int rows, C, KT, n0, m0;
  int4_t rsrc_a, rsrc_b;  // of operands that are contiguous along the contraction
};

// The output's rows of a big tile: a unit's, or BM rows of a group's dW.
struct GroupedRows {
  int group, begin, end;  // the group's rows of the operands
  int row;                // the first row of the output (of the group's dW in wgrad)
  int rows;               // and how many there are from there on
};

template <int OP>
__device__ inline GroupedTile grouped_tile(const GroupedArgs &a, const GroupedRows &g, int n0, int BM, int BN, int BK) {
  constexpr bool kTransA = OP == kGroupWgrad;
  constexpr bool kTransB = OP != kGroupForward;
  const int lda = OP == kGroupForward ? a.K : a.N;
  const int cols = OP == kGroupForward ? a.N : a.K;
  GroupedTile t{};
  t.n0 = n0;
  t.rows = min(BM, g.rows);
  if constexpr (OP != kGroupWgrad) {
    t.C = OP == kGroupForward ? a.K : a.N;
    t.pa = a.A + static_cast<int64_t>(g.row) * lda;
    t.pb = a.B + static_cast<int64_t>(g.group) * a.N * a.K;
    if constexpr (OP == kGroupForward) t.pb += static_cast<int64_t>(n0) * a.K;
    t.pd = a.D + static_cast<int64_t>(g.row) * cols;
  } else {
    t.m0 = g.row;
    t.C = g.end - g.begin;
    t.pa = a.A + static_cast<int64_t>(g.begin) * lda;
    t.pb = a.B + static_cast<int64_t>(g.begin) * a.K;
    t.pd = a.D + (static_cast<int64_t>(g.group) * a.N + g.row) * cols;
  }
  // A sum over nothing still walks one K tile, all of it out of range: zeros.
  t.KT = max(1, (t.C + BK - 1) / BK);
  if constexpr (!kTransA) t.rsrc_a = make_buffer_rsrc(t.pa, static_cast<uint32_t>(t.rows) * lda * 2u);
  if constexpr (!kTransB) t.rsrc_b = make_buffer_rsrc(t.pb, static_cast<uint32_t>(min(BN, cols - n0)) * a.K * 2u);
  return t;
}

// LDS of a phase: the ring, and behind it a block row of staging per wave, or
// (outputs whose rows are not aligned) the whole staged tile over the ring.
template <class S, bool ALIGNED>
constexpr int grouped_lds() {
  return ALIGNED ? S::kRingBytes + S::kWaves * 16 * S::kStagePitch : S::kLdsBytes;
}

// Computes the tiles that `next` gives, one after another: next(&tile) returns
// false when there are no more (both wave-uniform).  No other wave may still
// use the LDS, nor this one have loads to it in flight.
template <class S, int OP, bool ALIGNED, class Next>
__device__ __attribute__((always_inline)) inline void grouped_phase(const GroupedArgs &a, char *smem, Next next) {
  static_assert(S::MI == 16 && S::BK == 64 && S::STAGES >= 2 && S::SWIZZLE, "the pipelined 16x16x32 loop");
  constexpr bool kTransA = OP == kGroupWgrad;
  constexpr bool kTransB = OP != kGroupForward;

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / S::WAVES_N;
  const int wn = wave % S::WAVES_N;
  const uint32_t lds0 = lds_addr(smem);

  // Row strides (elements) of the operands, and the columns of the output.
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

  // The descriptor of K tile kt's rows of an operand that is not contiguous
  // along the contraction, from column `col0` on: rows past the contraction's
  // end read as zeros; columns past the operand's own only reach outputs that
  // are not stored.
  auto k_rows_rsrc = [&](const uint16_t *p, int ld, int col0, int C, int kt) {
    const int k0 = kt * S::BK;
    const int have = min(S::BK, C - k0);
    return make_buffer_rsrc(p + static_cast<int64_t>(k0) * ld + col0,
                            have > 0 ? static_cast<uint32_t>(have) * ld * 2u - static_cast<uint32_t>(col0) * 2u : 0u);
  };

  // This lane's byte offset in each operand, and the bytes from one load
  // instruction's rows to the next's; of a transposed operand every load's
  // offset (the flipped column is bit 6 of the element index).  Re-materialised
  // inside the tile loop, as in gemm_kernel.
  uint32_t off_a, step_a, trans_a[kTransA ? S::kDmaA : 1], trans_b[kTransB ? S::kDmaB : 1];
  int kcol;
  auto lane_offsets = [&]() {
    if constexpr (!kTransA) {
      off_a = static_cast<uint32_t>(ld_row) * lda * 2u + static_cast<uint32_t>(ld_kcol) * 2u;
      step_a = static_cast<uint32_t>(kRowStep) * lda * 2u;
      kcol = ld_kcol;
      asm volatile("" : "+v"(off_a), "+v"(kcol), "+s"(step_a));
    }
    auto trans = [&](auto tile, uint32_t row, uint32_t col, int ld, uint32_t *off) {
      using Tt = decltype(tile);
#pragma unroll
      for (int i = 0; i < S::BK / (Tt::kRowsPerDma * S::kWaves); ++i) {
        off[i] = ((row + static_cast<uint32_t>(i * Tt::kRowsPerDma * S::kWaves)) * static_cast<uint32_t>(ld) +
                  (flip(tile, i) ? col ^ 64u : col)) *
                 2u;
        asm volatile("" : "+v"(off[i]));
      }
    };
    if constexpr (kTransA) trans(TileA{}, ta_row, ta_col, lda, trans_a);
    if constexpr (kTransB) trans(TileB{}, tb_row, tb_col, ldb, trans_b);
  };

  struct DmaArgs {
    int4_t rsrc;
    uint32_t voffset;
  };
  // Load d of a K tile: descriptors ra and rb, and the K tile's first
  // contraction index (its byte offset and the range test of operands that
  // are contiguous along it).
  auto dma_args = [&](int4_t ra, int4_t rb, int C, int k0, int d) -> DmaArgs {
    const bool is_a = d < S::kDmaA;
    const int i = is_a ? d : d - S::kDmaA;
    if (is_a ? kTransA : kTransB) return DmaArgs{is_a ? ra : rb, is_a ? trans_a[i] : trans_b[i]};
    // Both operands' rows are equally long where neither is transposed.
    const uint32_t off = k0 + kcol < C ? off_a + static_cast<uint32_t>(k0) * 2u : kOobOffset;
    return DmaArgs{is_a ? ra : rb, off + static_cast<uint32_t>(i) * step_a};
  };
  auto lds_of = [&](int kt, int d) {
    const uint32_t at = lds0 + static_cast<uint32_t>((kt % S::STAGES) * S::kStageBytes) +
                        static_cast<uint32_t>(wave) * 1024u +
                        (d < S::kDmaA ? d * kLdsStep : S::kStageA + (d - S::kDmaA) * kLdsStep);
    return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(at));
  };
  auto load_of = [&](const GroupedTile &t, int kt, int d) {
    int4_t ra = t.rsrc_a, rb = t.rsrc_b;
    if (d < S::kDmaA) {
      if constexpr (kTransA) ra = k_rows_rsrc(t.pa, lda, t.m0, t.C, kt);
    } else {
      if constexpr (kTransB) rb = k_rows_rsrc(t.pb, ldb, t.n0, t.C, kt);
    }
    const DmaArgs g = dma_args(ra, rb, t.C, kt * S::BK, d);
    lds_dma_b128(g.rsrc, g.voffset, lds_of(kt, d));
  };
  auto load_ahead = [&](const GroupedTile &t) {
#pragma unroll
    for (int s = 0; s < grouped_ahead<S>(); ++s)
#pragma unroll
      for (int d = 0; d < S::kDmaPerStage; ++d) load_of(t, s, d);
  };

  GroupedTile cur;
  if (!next(&cur)) return;
  lane_offsets();
  load_ahead(cur);
  constexpr int kStores = S::kWaveM * S::kWaveN / 512;  // per wave and tile, 16 bytes a lane
  bool stores = false;
  for (;;) {
    lane_offsets();
    auto load_one = [&](int kt, int d) { load_of(cur, kt, d); };
    // Operand addresses, made new for every tile: what follows from them would
    // otherwise be worked out ahead of the tile loop and spilled across the
    // epilogue, and a spill's reload waits for every load in flight.  Of a
    // transposed operand all of them, in both stages of the early-free ring
    // (the second lies past the instruction's offset): worked out beside the
    // MFMAs they took issue slots (8192 rows x 4096 x 4096 wgrad 195 us).
    constexpr int kBases = S::EARLY_FREE ? 2 : 1;
    static_assert(!S::EARLY_FREE || S::STAGES == 2, "a base for each stage");
    uint32_t rd_a = a_row_base, rd_b = b_row_base, rd_swz = static_cast<uint32_t>(frag_kchunk ^ frag_swz) * 16;
    uint32_t rt_a[kBases][kTransA ? S::kFragM : 1], rt_b[kBases][kTransB ? S::kFragN : 1];
    if constexpr (!kTransA || !kTransB) asm volatile("" : "+v"(rd_a), "+v"(rd_b), "+v"(rd_swz));
#pragma unroll
    for (int st = 0; st < kBases; ++st) {
#pragma unroll
      for (int i = 0; i < (kTransA ? S::kFragM : 0); ++i) {
        rt_a[st][i] = (ta_base ^ (static_cast<uint32_t>(i) << 5)) + static_cast<uint32_t>(st * S::kStageBytes);
        asm volatile("" : "+v"(rt_a[st][i]));
      }
#pragma unroll
      for (int j = 0; j < (kTransB ? S::kFragN : 0); ++j) {
        rt_b[st][j] = (tb_base ^ (static_cast<uint32_t>(j) << 5)) + static_cast<uint32_t>(st * S::kStageBytes);
        asm volatile("" : "+v"(rt_b[st][j]));
      }
    }
    half8_t fa[2][S::kFragM], fb[2][S::kFragN];
    // Operand block `blk` of K step ks from the stage of K tile kt.
    auto read_block = [&](bool is_a, int blk, int kt, int ks) -> half8_t {
      const uint32_t stage = static_cast<uint32_t>((kt % S::STAGES) * S::kStageBytes);
      if (is_a ? kTransA : kTransB) {
        const uint32_t rb = is_a ? TileA::kRowBytes : TileB::kRowBytes;
        const int st = S::EARLY_FREE ? kt & 1 : 0;
        const uint32_t at = (is_a ? rt_a[st][blk] : rt_b[st][blk]) + (S::EARLY_FREE ? 0u : stage) +
                            static_cast<uint32_t>(ks) * 32u * rb;
        const half4_t lo = lds_read_transposed(at), hi = lds_read_transposed(at + 4 * rb);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
      // chunk (4 ks + frag_kchunk) ^ frag_swz of the row
      return *reinterpret_cast<const half8_t *>(smem + stage + (is_a ? rd_a : rd_b) + blk * 16 * S::kRowBytes +
                                                (rd_swz ^ static_cast<uint32_t>(ks * 64)));
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
      float zero = 0.0f;
      asm volatile("" : "+v"(zero));
#pragma unroll
      for (int i = 0; i < S::kFragM; ++i)
#pragma unroll
        for (int j = 0; j < S::kFragN; ++j) acc[i][j] = float4_t{zero, zero, zero, zero};
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
        rf_a = cur.rsrc_a;
        if constexpr (kTransA) rf_a = k_rows_rsrc(cur.pa, lda, cur.m0, cur.C, tile);
      } else if (part == 3) {
        rf_b = cur.rsrc_b;
        if constexpr (kTransB) rf_b = k_rows_rsrc(cur.pb, ldb, cur.n0, cur.C, tile);
      }
    };
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    auto mfma_load = [&](int buf, int idx, int tile, int d) {
      const int i = S::mfma_i(idx);
      const int j = S::mfma_j(idx);
      (void)tile;
      const DmaArgs g = dma_args(rf_a, rf_b, cur.C, rf_k0, d);
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
    using Base = KernelRingOps<S, decltype(mfma), decltype(read_frag), decltype(load_one), decltype(mfma_load),
                               decltype(prep), decltype(init_acc)>;
    GroupedRingOps<S, kStores, Base> ops{{mfma, read_frag, load_one, mfma_load, prep, init_acc}, false};
    // The loop's last barrier comes after every wave's last read of its
    // operands: the ring is free.
    grouped_k_loop<S>(ops, 0, cur.KT, stores);

    GroupedTile after{};
    const bool more = next(&after);
    if constexpr (ALIGNED) {
      if (more) {
        lane_offsets();
        load_ahead(after);
      }
    }

    // ---- epilogue ------------------------------------------------------------
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    // The lane, made new for every tile: the epilogue's addresses would
    // otherwise be worked out ahead of the tile loop and spilled.
    int ep_lane = lane;
    asm volatile("" : "+v"(ep_lane));
    const int ep_row = ep_lane % 16;
    const int ep_kgrp = ep_lane / 16;
    const int n = cur.n0 + wn * S::kWaveN;
    if constexpr (ALIGNED) {
      // A block row (16 rows) at a time through this wave's part of the
      // staging area behind the ring, which the loads above do not touch:
      // 8 bytes of a row per lane in, whole 16-byte pieces of consecutive
      // columns out.
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
          cur.pd, 0, static_cast<int>(static_cast<uint32_t>(cur.rows) * cols * 2u), 0x00020000);
      char *const tile = smem + S::kRingBytes + wave * 16 * S::kStagePitch;
      constexpr int kPieces = S::kWaveN / 8;
      constexpr int kPerPass = 64 / kPieces;
      const int c = n + ep_lane % kPieces * 8;
      const char *const from = tile + ep_lane / kPieces * S::kStagePitch + ep_lane % kPieces * 16;
      const int row0 = wm * S::kWaveM + ep_lane / kPieces;
#pragma unroll
      for (int i = 0; i < S::kFragM; ++i) {
        // Still in AGPRs here: the compiler would read all of them into VGPRs
        // ahead of the loads above.
#pragma unroll
        for (int j = 0; j < S::kFragN; ++j) asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
        for (int j = 0; j < S::kFragN; ++j) {
          half4_t h;
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = round_out<S::DTYPE>(acc[i][j][e]);
          *reinterpret_cast<half4_t *>(tile + ep_row * S::kStagePitch + (j * 16 + ep_kgrp * 4) * 2) = h;
        }
#pragma unroll
        for (int r = 0; r < 16; r += kPerPass) {
          const uint4_v v = *reinterpret_cast<const uint4_v *>(from + r * S::kStagePitch);
          const uint32_t off = c < cols ? static_cast<uint32_t>(row0 + i * 16 + r) * static_cast<uint32_t>(cols) * 2u +
                                              static_cast<uint32_t>(c) * 2u
                                        : kOobOffset;
          __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, static_cast<int>(off), 0, kStreamed);
        }
        __builtin_amdgcn_sched_barrier(0);  // a block row at a time, for the registers
      }
      stores = true;
    } else {
      wait_vmcnt<0>();  // the loads past the last K tile have written their zeros
      workgroup_barrier();
      char *const tile = smem + wave * S::kWaveM * S::kStagePitch;
#pragma unroll
      for (int i = 0; i < S::kFragM; ++i) {
#pragma unroll
        for (int j = 0; j < S::kFragN; ++j) asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
        for (int j = 0; j < S::kFragN; ++j) {
          half4_t h;
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = round_out<S::DTYPE>(acc[i][j][e]);
          *reinterpret_cast<half4_t *>(tile + (i * 16 + ep_row) * S::kStagePitch + (j * 16 + ep_kgrp * 4) * 2) = h;
        }
        __builtin_amdgcn_sched_barrier(0);  // a block row at a time, for the registers
      }
      _Float16 *const dst = reinterpret_cast<_Float16 *>(cur.pd) + static_cast<int64_t>(wm * S::kWaveM) * cols + n;
      store_wave_tile<S::kWaveM, S::kWaveN, S::kStagePitch>(tile, dst, cols, cur.rows - wm * S::kWaveM, cols - n,
                                                            a.alignment, ep_lane);
      __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
      workgroup_barrier();  // every wave has read its staged tile
      if (more) {
        lane_offsets();
        load_ahead(after);
      }
    }
    if (!more) break;
    cur = after;
  }
  // Nothing of this phase writes to the LDS any more: the loads past the last K
  // tile, which are older than the stores, have landed in every wave.
  wait_vmcnt<ALIGNED ? kStores : 0>();
  workgroup_barrier();
}

// Estimated time, in percent of a round of 256x256 tiles, of `n` of them on
// `grid` workgroups and `more` quarters, when a last round that would leave half
// of the workgroups or more without a tile (or any, if there are quarters
// anyway) is cut into quarters.  128x128 tiles have 71 % of the bigger ones'
// rate (8192x4096x2048 in one group: 137 us and 97.6 us).
__host__ __device__ inline int64_t big_rounds(int64_t n, int64_t more, int64_t grid) {
  const int64_t left = n % grid;
  if (more == 0 && 2 * left > grid) return 100 * (n / grid + 1);
  return 100 * (n / grid) + (4 * left + more + grid - 1) / grid * (100 * 25 / 71);
}

// S tiles in whole rounds of all workgroups.  With Q (a quarter of S; S itself
// for none), what would be a last round of few tiles is cut into quarters, and
// where it shortens the estimate so are the groups' last units that have no more
// than half their rows (at the end, where they read their group's weights
// again: 8200 rows over 16 groups x 4096 x 2048 149 -> 137 us).
template <class S, class Q, int OP, bool ALIGNED, int CAP>
__global__ void __launch_bounds__(S::kThreads) __attribute__((amdgpu_waves_per_eu(S::kWaves / 4, S::kWaves / 4)))
grouped_gemm_kernel(GroupedArgs a) {
  constexpr bool kQuarters = !std::is_same_v<S, Q>;
  static_assert(!kQuarters || (Q::BM * 2 == S::BM && Q::BN * 2 == S::BN && Q::kThreads == S::kThreads),
                "quarters of a tile");
  constexpr bool kUnits = OP != kGroupWgrad;
  // The table lies behind the rings in one allocation, so that the rings start
  // at LDS address 0 and their offsets fit the instructions.
  using Table = std::conditional_t<kUnits, GroupTable<CAP>, WgradTable<CAP>>;
  constexpr int kLds = ring_max(grouped_lds<S, ALIGNED>(), grouped_lds<Q, ALIGNED>());
  static_assert(kLds + sizeof(Table) <= 160 * 1024, "gfx950 has 160 KiB of LDS per CU");
  __shared__ __attribute__((aligned(1024))) char smem[kLds + sizeof(Table)];
  Table &table = *reinterpret_cast<Table *>(smem + kLds);

  const int cols = OP == kGroupForward ? a.N : a.K;
  const int tiles_n = (cols + S::BN - 1) / S::BN;
  const int tiles_m = (a.N + S::BM - 1) / S::BM;  // of a group's dW
  const int grid = static_cast<int>(gridDim.x);
  const int logical = static_cast<int>(xcd_logical_id(blockIdx.x, grid));
  int64_t num_tiles;
  if constexpr (kUnits) {
    build_group_table(&table, a.offsets, a.E, a.T, S::BM);
    __syncthreads();
    num_tiles = static_cast<int64_t>(table_units(&table, a.E)) * tiles_n;
  } else {
    build_wgrad_table(&table, a.offsets, a.E, a.T, S::kThreads);
    __syncthreads();
    num_tiles = static_cast<int64_t>(a.E) * tiles_m * tiles_n;
  }
  // The output rows and first column of big tile u.
  auto big_tile = [&](int64_t u, int *n0) -> GroupedRows {
    GroupedRows r;
    if constexpr (kUnits) {
      int tn;
      const GroupUnit g = table_tile(&table, a.E, S::BM, tiles_n, u, &tn);
      *n0 = tn * S::BN;
      r.group = g.group;
      r.row = g.row;
      r.rows = min(S::BM, g.end - g.row);
    } else {
      const int per = tiles_m * tiles_n;
      const int at = static_cast<int>(u / per);
      const TileCoord tc = tile_of(u - static_cast<int64_t>(at) * per, tiles_m, tiles_n, kGemmGroupM);
      *n0 = static_cast<int>(tc.tn) * S::BN;
      r.group = __builtin_amdgcn_readfirstlane(table.group[at]);
      r.begin = __builtin_amdgcn_readfirstlane(table.begin[at]);
      r.end = __builtin_amdgcn_readfirstlane(table.end[at]);
      r.row = static_cast<int>(tc.tm) * S::BM;
      r.rows = min(S::BM, a.N - r.row);
    }
    return r;
  };

  int lights = 0;  // units that are cut into quarters as well
  if constexpr (kUnits && kQuarters) {
    lights = table_light_units(&table, a.E, S::BM);
    const int64_t heavy = num_tiles - static_cast<int64_t>(lights) * tiles_n;
    const bool apart =
        big_rounds(heavy, 2 * static_cast<int64_t>(lights) * tiles_n, grid) < big_rounds(num_tiles, 0, grid);
    lights = __builtin_amdgcn_readfirstlane(apart ? lights : 0);
    num_tiles -= static_cast<int64_t>(lights) * tiles_n;
    __syncthreads();
    if (lights > 0) table_drop_light(&table, a.E, S::BM);
    __syncthreads();
  }
  const int64_t whole = num_tiles / grid;
  const int left = static_cast<int>(num_tiles - whole * grid);
  const bool quarters = kQuarters && (lights > 0 || 2 * left <= grid);
  const int64_t rounds = quarters ? whole : whole + 1;
  int64_t round = 0;
  grouped_phase<S, OP, ALIGNED>(a, smem, [&](GroupedTile *t) {
    if (round == rounds) return false;
    // Forwards; in wgrad backwards in every other round.
    const int64_t u = round * grid + (!kUnits && (round & 1) ? grid - 1 - logical : logical);
    ++round;
    if (u >= num_tiles) return false;  // only the last round is not whole
    int n0;
    const GroupedRows r = big_tile(u, &n0);
    *t = grouped_tile<OP>(a, r, n0, S::BM, S::BN, S::BK);
    return true;
  });
  if constexpr (!kQuarters) return;
  if (!quarters) return;
  // Upper halves first, so that halves without rows come last; then the light
  // units' only halves.
  const int64_t all = 4 * left + 2 * static_cast<int64_t>(lights) * tiles_n;
  int64_t at = logical;
  grouped_phase<Q, OP, ALIGNED>(a, smem, [&](GroupedTile *t) {
    for (; at < all; at += grid) {
      if constexpr (kUnits) {
        if (at >= 4 * left) {
          const int rest = static_cast<int>(at - 4 * left);
          const int k = rest / (2 * tiles_n);
          const int n0 = (rest - k * 2 * tiles_n) * Q::BN;
          if (n0 >= cols) continue;
          const GroupUnit g = table_light_unit(&table, a.E, S::BM, k);
          GroupedRows r{};
          r.group = g.group;
          r.row = g.row;
          r.rows = g.end - g.row;
          *t = grouped_tile<OP>(a, r, n0, Q::BM, Q::BN, Q::BK);
          at += grid;
          return true;
        }
      }
      const int s = static_cast<int>(at);
      const int low = s >= 2 * left;
      const int rest = s - low * 2 * left;
      int n0;
      GroupedRows r = big_tile(whole * grid + rest / 2, &n0);
      r.row += low * Q::BM;
      r.rows -= low * Q::BM;
      n0 += rest % 2 * Q::BN;
      if (r.rows <= 0 || n0 >= cols) continue;
      *t = grouped_tile<OP>(a, r, n0, Q::BM, Q::BN, Q::BK);
      at += grid;
      return true;
    }
    return false;
  });
}

// The tile (of kTile256x256, which stands for it with quarters, kTile256x128
// and kTile128x128) with the least estimated time in rounds of all CUs.  The
// smaller ones' rates of the 256x256 one are measured (8192x4096x2048 in one
// group: 97.6 us, 127 and 137 us).
constexpr int kGroupedCap = 512;  // groups the 256x128 tile's ring leaves room for
inline GemmTile grouped_default_tile(int op, int64_t T, int64_t N, int64_t K, int64_t E, int num_cus) {
  const int64_t cols = op == kGroupForward ? N : K;
  auto tiles = [&](int64_t bm, int64_t bn) {
    return (op == kGroupWgrad ? E * ((N + bm - 1) / bm) : expected_units(T, E, bm)) * ((cols + bn - 1) / bn);
  };
  auto rounds = [&](int64_t n) { return (n + num_cus - 1) / num_cus; };
  // Times in percent of a round of 256x256 tiles.
  const int64_t small = 100 * rounds(tiles(128, 128)) * 25 / 71;
  const int64_t mid = 100 * rounds(tiles(256, 128)) * 50 / 77;
  int64_t big = big_rounds(tiles(256, 256), 0, num_cus);
  if (op != kGroupWgrad) {
    // Half the groups' last units are light.
    const int64_t across = (cols + 255) / 256;
    const int64_t apart = big_rounds(T / 256 * across, (E < T ? E : T) * across, num_cus);
    big = apart < big ? apart : big;
  }
  if (big < small && (big <= mid || E > kGroupedCap)) return kTile256x256;
  return mid < small && E <= kGroupedCap ? kTile256x128 : kTile128x128;
}

template <class S, class Q, int OP, int CAP>
static hipError_t launch_grouped_shape(const GroupedArgs &a, int num_cus, hipStream_t stream) {
  const int cols = OP == kGroupForward ? a.N : a.K;
  // No more workgroups than there can be tiles, or quarters of tiles.
  const int64_t down =
      OP == kGroupWgrad ? static_cast<int64_t>(a.E) * ((a.N + S::BM - 1) / S::BM) : unit_bound(a.T, a.E, S::BM);
  const int64_t tiles = (std::is_same_v<S, Q> ? 1 : 4) * down * ((cols + S::BN - 1) / S::BN);
  const dim3 grid(static_cast<unsigned>(tiles < num_cus ? tiles : num_cus));
  // The gradients' rows are a multiple of 8 elements long, and their outputs
  // 16-byte aligned.
  if (OP != kGroupForward || a.alignment == 16)
    hipLaunchKernelGGL((grouped_gemm_kernel<S, Q, OP, true, CAP>), grid, dim3(S::kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((grouped_gemm_kernel<S, Q, OP, OP != kGroupForward, CAP>), grid, dim3(S::kThreads), 0, stream, a);
  return hipGetLastError();
}

template <int DT, int OP>
static hipError_t launch_grouped_op(const void *A, const void *B, const int *offsets, void *D, int T, int N, int K, int E,
                                    int num_cus, hipStream_t stream) {
  using Big = std::conditional_t<DT == kF16, GemmDefault, GemmBf16>;
  using Mid = GemmTile256x128<DT, kGemmTileShapes[kTile256x128].stages>;
  using Small = GemmTile128x128<DT, kGemmTileShapes[kTile128x128].stages>;
  const GroupedArgs a{static_cast<const uint16_t *>(A), static_cast<const uint16_t *>(B), static_cast<uint16_t *>(D),
                      offsets, T, N, K, E, row_alignment(D, OP == kGroupForward ? N : K)};
  switch (grouped_default_tile(OP, T, N, K, E, num_cus)) {
    case kTile256x128: return launch_grouped_shape<Mid, Mid, OP, kGroupedCap>(a, num_cus, stream);
    case kTile128x128: return launch_grouped_shape<Small, Small, OP, kMaxGroups>(a, num_cus, stream);
    default: return launch_grouped_shape<Big, Small, OP, kMaxGroups>(a, num_cus, stream);
  }
}

}  // namespace gt
