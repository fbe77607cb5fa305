// grouped_wgrad.hip -- the grouped product dW[e, n, k] = sum_t dY[t, n] X[t, k]
// on the tiled kernel of grouped_kernel.hpp.
#include "grouped_kernel.hpp"

namespace gt {

hipError_t launch_grouped_wgrad(int dtype, const void *A, const void *B, const int *offsets, void *D, int T, int N, int K,
                                int E, int num_cus, hipStream_t stream) {
  return dtype == kBF16 ? launch_grouped_op<kBF16, kGroupWgrad>(A, B, offsets, D, T, N, K, E, num_cus, stream)
                        : launch_grouped_op<kF16, kGroupWgrad>(A, B, offsets, D, T, N, K, E, num_cus, stream);
}

}  // namespace gt
