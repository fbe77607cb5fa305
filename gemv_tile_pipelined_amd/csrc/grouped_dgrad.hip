// grouped_dgrad.hip -- the grouped product dX[t, k] = sum_n dY[t, n] W[e, n, k]
// on the tiled kernel of grouped_kernel.hpp.
#include "grouped_kernel.hpp"

namespace gt {

hipError_t launch_grouped_dgrad(int dtype, const void *A, const void *B, const int *offsets, void *D, int T, int N, int K,
                                int E, int num_cus, hipStream_t stream) {
  return dtype == kBF16 ? launch_grouped_op<kBF16, kGroupDgrad>(A, B, offsets, D, T, N, K, E, num_cus, stream)
                        : launch_grouped_op<kF16, kGroupDgrad>(A, B, offsets, D, T, N, K, E, num_cus, stream);
}

}  // namespace gt
