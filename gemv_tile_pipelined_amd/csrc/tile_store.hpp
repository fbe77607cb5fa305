// tile_store.hpp -- how the grouped and the 8-bit tiled kernels write a wave's
// output tile, which they have staged in LDS row by row as 16-bit numbers.
#pragma once

#include "device_common.hpp"

namespace gt {

// Bytes by which every row of an output of `ld` columns at D is aligned: 16, 4
// or 2.
inline int row_alignment(const void *D, int64_t ld) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(D);
  return ld % 8 == 0 && at % 16 == 0 ? 16 : ld % 2 == 0 && at % 4 == 0 ? 4 : 2;
}

// Writes the first `rows` rows and `cols` columns of a ROWS x COLS tile staged
// at `tile` (PITCH bytes a row) to `dst` (`ld` elements a row).
//
// 16-byte aligned rows leave in whole 16-byte pieces, 8 elements a lane, with
// non-temporal stores (gemm_kernel.hpp).  Others leave in aligned pairs, one a
// lane and so consecutive over the lanes (cached: neighbouring tiles' rows
// share lines), and every second row of an odd number of columns has a single
// element at either end.  8192 rows over 16 groups x 4095 (4094) x 2048 take 173
// (162) us beside 154 for 4096 columns; stored 8 elements a lane one by one it
// was 1 % more than in pairs, one element a lane 9 %, and 16-byte pieces of rows
// staged shifted by their misalignment were level for odd and 9 % more for even
// numbers of columns.
template <int ROWS, int COLS, int PITCH>
__device__ inline void store_wave_tile(const char *tile, _Float16 *dst, int64_t ld, int rows, int cols, int alignment,
                                       int lane) {
  static_assert(COLS == 32 || COLS == 64 || COLS == 128, "tile columns");
  if (alignment == 16) {
    constexpr int kPieces = COLS / 8;
    constexpr int kPerPass = 64 / kPieces;
    const int n = lane % kPieces * 8;
#pragma unroll 4
    for (int r0 = 0; r0 < ROWS; r0 += kPerPass) {
      const int r = r0 + lane / kPieces;
      const half8_t v = *reinterpret_cast<const half8_t *>(tile + r * PITCH + n * 2);
      if (r < rows && n < cols)  // columns come in eights
        __builtin_nontemporal_store(v, reinterpret_cast<half8_t *>(dst + r * ld + n));
    }
    return;
  }
  constexpr int kPerPass = 128 / COLS;
  const int pair = lane % (COLS / 2) * 2;
  if (alignment == 4) {
#pragma unroll 8
    for (int r0 = 0; r0 < ROWS; r0 += kPerPass) {
      const int r = r0 + lane / (COLS / 2);
      const half2_t v = *reinterpret_cast<const half2_t *>(tile + r * PITCH + pair * 2);
      if (r < rows && pair < cols) *reinterpret_cast<half2_t *>(dst + r * ld + pair) = v;
    }
    return;
  }
  const int have = min(cols, COLS);
  auto odd = [&](const _Float16 *row) { return static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1) & 1; };
#pragma unroll 8
  for (int r0 = 0; r0 < ROWS; r0 += kPerPass) {
    const int r = r0 + lane / (COLS / 2);
    _Float16 *row = dst + r * ld;
    const int n = pair - odd(row);  // a row that starts on the upper half of a word pairs from its second element
    const _Float16 *at = reinterpret_cast<const _Float16 *>(tile + r * PITCH) + max(n, 0);
    const half2_t v = {at[0], at[1]};
    if (r < rows && n >= 0 && n + 1 < have) *reinterpret_cast<half2_t *>(row + n) = v;
  }
#pragma unroll
  for (int r0 = 0; r0 < ROWS; r0 += 32) {  // the single elements: first and last of 32 rows
    const int r = r0 + lane / 2;
    _Float16 *row = dst + r * ld;
    const int first = odd(row);
    const int n = lane & 1 ? have - 1 : 0;
    const bool single = lane & 1 ? ((have - first) & 1) != 0 : first != 0;
    if (r < min(rows, ROWS) && have > 0 && single) row[n] = reinterpret_cast<const _Float16 *>(tile + r * PITCH)[n];
  }
}

}  // namespace gt
