// groups.hpp -- which rows of which group a workgroup of a grouped product
// computes.
//
// A grouped product has T rows sorted by group and an array offsets[E + 1] in
// device memory: group e owns rows offsets[e] .. offsets[e + 1] - 1.  A
// kernel cuts every group's rows into blocks of `rows` ("units"), counted
// group by group; the number of units is known on the device only, so the
// host launches unit_bound() of them and those past the last return at once.
//
// The offsets are not read by the host (that would need a synchronisation),
// so they are made safe where they are read: a group's rows are
// [begin, end) with begin = offsets[e] clamped to [0, T] and end =
// offsets[e + 1] clamped to [begin, T].  No value of offsets lets a kernel
// read or write outside the T rows.  (With offsets that are not
// non-decreasing the units may outnumber the bound, and then the last ones
// are not computed.)
#pragma once

#include <stdint.h>

#include "tile_order.hpp"  // GT_HD

namespace gt {

// Most groups of a grouped product: the tiled kernels keep a table of the
// groups in LDS.
constexpr int kMaxGroups = 1024;

struct GroupRows {
  int begin;
  int end;
};

GT_HD inline GroupRows group_rows(int first, int next, int T) {
  GroupRows g;
  g.begin = first < 0 ? 0 : (first > T ? T : first);
  g.end = next < g.begin ? g.begin : (next > T ? T : next);
  return g;
}

// First row of a group's unit `at`, which offsets that are not non-decreasing can
// make any number (the count of units may then overflow): kept in the group.
GT_HD inline int unit_row(GroupRows g, int at, int rows) {
  const int64_t row = g.begin + static_cast<int64_t>(at) * rows;
  return row < g.begin ? g.begin : row > g.end ? g.end : static_cast<int>(row);
}

// No more units than this for T rows in E groups: every group's last unit may
// be short, and no more groups than rows have any.
GT_HD inline int64_t unit_bound(int64_t T, int64_t E, int64_t rows) {
  const int64_t some = E < T ? E : T;
  return (T - some) / rows + some;
}

// Units of `rows` rows to expect for T rows in E groups whose sizes are not
// known on the host: T / rows whole ones, and half a unit more for each group
// that can have rows; but one at least for each of these.
inline int64_t expected_units(int64_t T, int64_t E, int64_t rows) {
  const int64_t some = E < T ? E : T;
  const int64_t units = T / rows + (some + 1) / 2;
  const int64_t bound = unit_bound(T, E, rows);
  return units < some ? some : units < bound ? units : bound;
}

// Whether the groups are streamed (stream.hip) in units of kStreamUnit rows, by
// the mean rows of a group, or tiled.  Measured (bf16, us streamed and tiled):
// 32 groups x 2048 x 2048 with a mean of 4 rows 51 and 62, 8 rows 58 and 66, 12
// rows 65 and 66, 16 rows 74 and 67, 32 rows 113 and 67; 8 bits, 64 groups x
// 2048 x 4096: 97 and 120, 107 and 121, 113 and 121, 121 and 120, 202 and 115.
constexpr int kStreamUnit = 16;
inline bool grouped_streams(int64_t T, int64_t N, int64_t E) {
  // A grid's threads are counted in 32 bits.
  return T <= 8 * E && unit_bound(T, E, kStreamUnit) * ((N + 15) / 16) < (int64_t{1} << 22);
}

}  // namespace gt

#if defined(__HIPCC__)
namespace gt {

struct GroupUnit {
  int group;
  int row;  // first row of the unit
  int end;  // end of its group's rows
};

// Inclusive sum over the lanes of a wave.
__device__ inline int wave_scan(int v) {
  const int lane = static_cast<int>(threadIdx.x & 63);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(v, d);
    if (lane >= d) v += up;
  }
  return v;
}

// Unit `u` of the groups cut into `rows` rows each; false past the last unit.
// Every wave of a workgroup works it out for itself (one read of the offsets
// from the caches for every 256 groups, and a scan): cheaper for a short
// kernel than a launch of its own or a barrier.  u is wave-uniform, and all
// 64 lanes must be active.
__device__ inline bool find_unit(const int *__restrict__ offsets, int E, int T, int rows, int u, GroupUnit *out) {
  constexpr int kAhead = 4;
  const int lane = static_cast<int>(threadIdx.x & 63);
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64 * kAhead) {
    int first[kAhead], next[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int e = e0 + 64 * j + lane;
      first[j] = e < E ? offsets[e] : T;  // groups past the last are empty
      next[j] = e < E ? offsets[e + 1] : T;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const GroupRows g = group_rows(first[j], next[j], T);
      const int n = (g.end - g.begin + rows - 1) / rows;
      const int upto = before + wave_scan(n);
      const uint64_t past = __ballot(upto > u);
      if (past != 0) {
        const int l = __builtin_ctzll(past);
        const int at = u - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(n, l));
        out->group = e0 + 64 * j + l;
        const GroupRows its{__builtin_amdgcn_readlane(g.begin, l), __builtin_amdgcn_readlane(g.end, l)};
        out->row = unit_row(its, at, rows);
        out->end = its.end;
        return true;
      }
      before = __builtin_amdgcn_readlane(upto, 63);
    }
  }
  return false;
}

constexpr int kUnitsAcross = 8;  // units that a column of tiles runs through before the next (as kGemmGroupM)

// The groups' units as a table in LDS, for persistent kernels that look up
// one unit after another.  CAP: the most groups it holds.
template <int CAP>
struct GroupTable {
  int upto[CAP];       // units of groups 0 .. e
  int begin[CAP + 1];  // rows of group e: begin[e] .. max(begin[e], begin[e + 1]) - 1
};

// Fills the table (the first wave of the workgroup; the caller places a
// barrier before the first use).
template <int CAP>
__device__ inline void build_group_table(GroupTable<CAP> *table, const int *__restrict__ offsets, int E, int T, int rows) {
  if (threadIdx.x >= 64) return;
  const int lane = static_cast<int>(threadIdx.x);
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    const GroupRows g = group_rows(e < E ? offsets[e] : T, e < E ? offsets[e + 1] : T, T);
    const int upto = before + wave_scan((g.end - g.begin + rows - 1) / rows);
    if (e < E) {
      table->upto[e] = upto;
      table->begin[e] = g.begin;
    }
    if (e == E - 1) table->begin[E] = g.end;
    before = __builtin_amdgcn_readlane(upto, 63);
  }
}

// Groups whose last unit has no more than half its rows ("light").
template <int CAP>
__device__ inline bool table_is_light(const GroupTable<CAP> *table, int E, int rows, int e) {
  if (e >= E) return false;
  const int tail = max(0, table->begin[e + 1] - table->begin[e]) % rows;
  return tail != 0 && tail <= rows / 2;
}

template <int CAP>
__device__ inline int table_light_units(const GroupTable<CAP> *table, int E, int rows) {
  const int lane = static_cast<int>(threadIdx.x & 63);
  int n = 0;
  for (int e0 = 0; e0 < E; e0 += 64) n += __popcll(__ballot(table_is_light(table, E, rows, e0 + lane)));
  return n;
}

// Takes the light units out of the table (the first wave; barriers as for
// build_group_table).
template <int CAP>
__device__ inline void table_drop_light(GroupTable<CAP> *table, int E, int rows) {
  if (threadIdx.x >= 64) return;
  const int lane = static_cast<int>(threadIdx.x);
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    const int len = e < E ? max(0, table->begin[e + 1] - table->begin[e]) : 0;
    const int upto = before + wave_scan((len + rows - 1 - rows / 2) / rows);
    if (e < E) table->upto[e] = upto;
    before = __builtin_amdgcn_readlane(upto, 63);
  }
}

// Light unit `k` (wave-uniform, below table_light_units()).
template <int CAP>
__device__ inline GroupUnit table_light_unit(const GroupTable<CAP> *table, int E, int rows, int k) {
  const int lane = static_cast<int>(threadIdx.x & 63);
  int e = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    uint64_t light = __ballot(table_is_light(table, E, rows, e0 + lane));
    const int n = __popcll(light);
    if (k < n) {
      for (; k > 0; --k) light &= light - 1;
      e = e0 + __builtin_ctzll(light);
      break;
    }
    k -= n;
  }
  const int begin = table->begin[e], end = table->begin[e + 1];
  GroupUnit g;
  g.group = __builtin_amdgcn_readfirstlane(e);
  g.row = __builtin_amdgcn_readfirstlane(begin + (end - begin) / rows * rows);
  g.end = __builtin_amdgcn_readfirstlane(end);
  return g;
}

template <int CAP>
__device__ inline int table_units(const GroupTable<CAP> *table, int E) {
  return __builtin_amdgcn_readfirstlane(table->upto[E - 1]);
}

// Tile `u` (wave-uniform) of the table's units times `tiles_n` columns of tiles:
// its unit, and its column in *tn.  Group by group, and within a group in the
// grouped order of tile_order.hpp: the tiles that run side by side on an XCD then
// read the weights of a group or two, and most of each group's rows on one XCD
// only.  Against 8 units side by side whatever their groups: 16384 rows over 32
// groups x 4096 x 4096 515 -> 495 us in bf16, 305 -> 294 in 8 bits, dgrad of 8192
// over 16 x 4096 x 2048 147 -> 141.
template <int CAP>
__device__ inline GroupUnit table_tile(const GroupTable<CAP> *table, int E, int rows, int tiles_n, int64_t u, int *tn) {
  const int lane = static_cast<int>(threadIdx.x & 63);
  const int unit = static_cast<int>(u / tiles_n);  // counted unit by unit: of the same group
  int e = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const uint64_t past = __ballot(e0 + lane < E && table->upto[e0 + lane < E ? e0 + lane : 0] > unit);
    if (past != 0) {
      e = e0 + __builtin_ctzll(past);
      break;
    }
  }
  const int before = __builtin_amdgcn_readfirstlane(e > 0 ? table->upto[e - 1] : 0);
  const int units = __builtin_amdgcn_readfirstlane(table->upto[e]) - before;
  const int begin = __builtin_amdgcn_readfirstlane(table->begin[e]);
  const int next = __builtin_amdgcn_readfirstlane(table->begin[e + 1]);
  const TileCoord tc = tile_of(u - static_cast<int64_t>(before) * tiles_n, units, tiles_n, kUnitsAcross);
  *tn = static_cast<int>(tc.tn);
  const GroupRows its{begin, next < begin ? begin : next};
  return GroupUnit{__builtin_amdgcn_readfirstlane(e), unit_row(its, static_cast<int>(tc.tm), rows), its.end};
}

}  // namespace gt
#endif
