// grouped_forward.hip -- the grouped product D[t, n] = sum_k X[t, k] W[e, n, k]
// on the tiled kernel of grouped_kernel.hpp.
#include "grouped_kernel.hpp"

namespace gt {

hipError_t launch_grouped_forward(int dtype, const void *A, const void *B, const int *offsets, void *D, int T, int N, int K,
                                int E, int num_cus, hipStream_t stream) {
  return dtype == kBF16 ? launch_grouped_op<kBF16, kGroupForward>(A, B, offsets, D, T, N, K, E, num_cus, stream)
                        : launch_grouped_op<kF16, kGroupForward>(A, B, offsets, D, T, N, K, E, num_cus, stream);
}

void grouped_plan_tile(int op, int64_t T, int64_t N, int64_t K, int64_t E, int num_cus, int *rows, int *cols) {
  const GemmTileShape &s = kGemmTileShapes[grouped_default_tile(op, T, N, K, E, num_cus)];
  *rows = s.bm;
  *cols = s.bn;
}

}  // namespace gt
