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

// The grouped K loop, recorded instead of run.
namespace {
template <class S>
struct GroupedRecorder : RingRecorder<S> {
  void wait_first(bool) { this->push(kRingWaitTile, GroupedWaits<S>::kFirst); }
  void wait_tile(int n) { this->push(kRingWaitTile, GroupedWaits<S>::in_loop(n)); }
};

template <class S>
int64_t record_grouped(int first, int ktu, int32_t *events, int64_t cap, int *info) {
  info[0] = S::kDmaPerStage;
  info[1] = S::STAGES;
  info[2] = grouped_ahead<S>();
  GroupedRecorder<S> rec{{S::STAGES, events, cap}};
  grouped_k_loop<S>(rec, first, ktu, false);
  return rec.n;
}
}  // namespace

int64_t grouped_ring_trace(int rows, int cols, int first, int ktu, int32_t *events, int64_t cap, int *info) {
  if (rows == 256 && cols == 256) return record_grouped<GemmDefault>(first, ktu, events, cap, info);
  if (rows == 256 && cols == 128)
    return record_grouped<GemmTile256x128<kF16, kGemmTileShapes[kTile256x128].stages>>(first, ktu, events, cap, info);
  if (rows == 128 && cols == 128)
    return record_grouped<GemmTile128x128<kF16, kGemmTileShapes[kTile128x128].stages>>(first, ktu, events, cap, info);
  return -1;
}

}  // namespace gt
