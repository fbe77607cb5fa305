// route.hip -- which experts a token goes to, with what weights, in which rows;
// and the gradient of the weights.
//
//   score[e]  = softmax over e of logit, or sigmoid(logit)
//   choice[e] = score[e] + bias[e], or logit[e] without a bias (scores are ordered as logits are)
//   groups of E / G experts: a group counts by its best choice, or the sum of its
//   two best; the best of the groups are kept
//   ids       = the k largest choices in kept groups, largest first, ties to the lowest index
//   weights   = scale * score[id], over their sum if they are normalised
//
// One wave has one token, its lanes V experts each that follow one another (V a
// power of two).  A choice becomes an unsigned key that orders as the numbers do
// (NaN below all of them), so that one of the k rounds is a maximum over the lane's
// keys, a maximum over the wave through DPP, and a ballot: the lowest lane that
// has the maximum has the lowest index.
//
// Ids are those of exact arithmetic.  Logits are compared as they are; where
// scores matter (a bias, or sums of two) they are computed in FP32 and every
// decision (each choice against the next, the last kept group against the first
// dropped) is checked against the error that these can have; a token with a
// closer decision, few in ten thousand of random ones, is done again in FP64.
#include "device_common.hpp"
#include "../../include/gemvtile.h"
#include "kernels.hpp"
#include "wave_ops.hpp"

namespace gt {

namespace {

constexpr int kWaves = 4;  // tokens of a workgroup
constexpr float kNegInf = -__builtin_inff();

// What FP32 choices can be off.  Exponentials and quotients lose a few units of
// 2^-24 each and a sum over E <= 1024 scores, added in a tree of 4 + 6 levels, at
// most 10 more: 2^-20 of the token's largest score bounds every score.  Adding a
// bias rounds by 2^-24 of the choice.  A choice x that is far below in FP32 cannot
// be ahead of c in truth, however large it is: it would take |x| within 2^-22 of
// |c|.  The bounds below are twice what that takes.
__device__ inline float choice_margin(float top_score, float a, float b) {
  return 0x1p-18f * top_score + 0x1p-22f * (__builtin_fabsf(a) + __builtin_fabsf(b));
}
// The same of a group's one or two best.
__device__ inline float group_error(float top_score, float first, float second) {
  return 0x1p-18f * top_score + 0x1p-22f * (__builtin_fabsf(first) + __builtin_fabsf(second));
}

// ---- keys --------------------------------------------------------------------
template <typename F>
struct KeyOf;
template <>
struct KeyOf<float> {
  typedef uint32_t type;
  static __device__ inline uint32_t of(float v) {
    if (v != v) return 1u;
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);  // -0 counts as 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;              // -inf: 0x007fffff
  }
  // The number of a key (a NaN's becomes NaN).
  static __device__ inline float value(uint32_t k) {
    return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7fffffffu : ~k);
  }
};
template <>
struct KeyOf<double> {
  typedef uint64_t type;
  static __device__ inline uint64_t of(double v) {
    if (v != v) return 1u;
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    return b >> 63 ? ~b : b | (uint64_t{1} << 63);
  }
};
// Key 0: no expert, or one taken or of a group that is not kept.

using gt::wave_max;
__device__ inline uint64_t wave_max(uint64_t v) {
#pragma unroll
  for (int lane = 1; lane < 64; lane <<= 1) {
    const uint64_t o = static_cast<uint64_t>(__shfl_xor(static_cast<unsigned long long>(v), lane));
    v = o > v ? o : v;
  }
  return v;
}
__device__ inline float wave_add(float v) { return wave_sum(v); }
__device__ inline double wave_add(double v) {
#pragma unroll
  for (int lane = 1; lane < 64; lane <<= 1) v += __shfl_xor(v, lane);
  return v;
}
__device__ inline float wave_max_logit(float v) {  // NaN left aside
  return KeyOf<float>::value(wave_max(KeyOf<float>::of(v == v ? v : kNegInf)));
}

// ---- logits --------------------------------------------------------------------
template <int DT>
struct Element {
  typedef uint16_t type;
};
template <>
struct Element<kF32> {
  typedef float type;
};
template <int DT>
__device__ inline float widen_logit(typename Element<DT>::type v) {
  if constexpr (DT == kF32) return v;
  else return widen_in<DT>(v);
}
template <int DT>
__device__ inline typename Element<DT>::type round_logit(float v) {
  if constexpr (DT == kF32) return v;
  else return __builtin_bit_cast(uint16_t, round_out<DT>(v));
}

// The lane's V logits of a row; -inf behind the last expert.  Rows are V * size
// apart from one another's alignment where E % V == 0: one load then.
template <int DT, int V>
__device__ inline void load_logits(const typename Element<DT>::type *row, int E, int lane, float *out) {
  typedef typename Element<DT>::type T;
  const int e0 = lane * V;
  if (E % V == 0) {
    if (e0 < E) {
      T v[V];
      __builtin_memcpy(v, __builtin_assume_aligned(row + e0, V * sizeof(T) < 16 ? V * sizeof(T) : 16), sizeof(v));
#pragma unroll
      for (int i = 0; i < V; ++i) out[i] = widen_logit<DT>(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) out[i] = kNegInf;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = e0 + i < E ? widen_logit<DT>(row[e0 + i]) : kNegInf;
  }
}

template <typename F>
__device__ inline F exp_of(F v) {
  if constexpr (sizeof(F) == 8) return ::exp(v);
  else return ::expf(v);
}
template <typename F>
__device__ inline F sigmoid(F v) {
  if (v < 0) {
    const F e = exp_of(v);
    return e / (1 + e);
  }
  return 1 / (1 + exp_of(-v));
}

// ---- the choice, in F --------------------------------------------------------
struct TopkArgs {
  int E, k, groups, top_groups, group_best, score, norm;
  float scale;
};

// The choice of one token: lane j < k gets the id of its j-th expert, lane k that
// of the best one left (-1 if there is none).  `buf` holds E numbers of the
// wave's own.  Returns whether a group was kept by a margin that FP32 does not
// vouch for (F = float).
template <typename F, int V>
__device__ inline bool choose(const float *logit, const float *bias, const TopkArgs &a, int lane, F *buf, int *id) {
  typedef typename KeyOf<F>::type Key;
  const bool ranked_by_logit = bias == nullptr;
  const bool scores = !ranked_by_logit || (a.groups > 1 && a.group_best == 2);
  F top_score = 1;  // at least the largest score
  F score[V];
  F choice[V];
  if (scores) {
    if (a.score == GEMVTILE_SCORE_SOFTMAX) {
      float m = kNegInf;
#pragma unroll
      for (int i = 0; i < V; ++i) m = logit[i] > m ? logit[i] : m;
      m = wave_max_logit(m);
      F sum = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        score[i] = m == kNegInf && logit[i] == kNegInf ? 0 : exp_of(static_cast<F>(logit[i]) - static_cast<F>(m));
        sum += score[i];
      }
      sum = wave_add(sum);
      if (sum == 0) sum = 1;  // every logit is -inf
      top_score = 1 / sum;
#pragma unroll
      for (int i = 0; i < V; ++i) score[i] /= sum;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) score[i] = sigmoid(static_cast<F>(logit[i]));
    }
  }
  Key key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    choice[i] = ranked_by_logit ? static_cast<F>(logit[i]) : score[i] + static_cast<F>(e < a.E ? bias[e] : 0.0f);
    key[i] = e < a.E ? KeyOf<F>::of(choice[i]) : 0;
  }
  bool close = false;
  if (a.groups > 1) {
    const int size = a.E / a.groups;
    const bool sums = a.group_best == 2 && size > 1;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane * V + i < a.E) buf[lane * V + i] = sums ? (ranked_by_logit ? score[i] : choice[i]) : choice[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    // Lane g works out group g.
    F value = 0;
    Key gkey = 0;
    float error = 0.0f;
    if (lane < a.groups) {
      F first = buf[lane * size], second = 0;
      Key k1 = KeyOf<F>::of(first), k2 = 0;
      for (int i = 1; i < size; ++i) {
        const F v = buf[lane * size + i];
        const Key kv = KeyOf<F>::of(v);
        if (kv > k1) {
          second = first;
          k2 = k1;
          first = v;
          k1 = kv;
        } else if (kv > k2) {
          second = v;
          k2 = kv;
        }
      }
      value = sums ? first + second : first;
      if (!sums) second = 0;
      if constexpr (sizeof(F) == 4) error = group_error(top_score, first, second);
      gkey = KeyOf<F>::of(value);
    }
    int rank = 0;  // groups ahead of this one
    for (int o = 0; o < a.groups; ++o) {
      Key other;
      if constexpr (sizeof(Key) == 8)
        other = static_cast<Key>(__shfl(static_cast<unsigned long long>(gkey), o));
      else
        other = static_cast<Key>(__builtin_amdgcn_readlane(static_cast<int>(gkey), o));
      rank += other > gkey || (other == gkey && o < lane) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < a.groups && rank < a.top_groups);
    if constexpr (sizeof(F) == 4) {
      // The last kept group against the first dropped one.
      if (scores && a.top_groups < a.groups) {
        const int last = __builtin_ctzll(__ballot(lane < a.groups && rank == a.top_groups - 1));
        const int next = __builtin_ctzll(__ballot(lane < a.groups && rank == a.top_groups));
        const float v1 = __shfl(value, last), v2 = __shfl(value, next);
        // The largest error of any group (as bits; a NaN above all).
        const float most = __builtin_bit_cast(float, wave_max(__builtin_bit_cast(uint32_t, error)));
        close = !(v1 - v2 > 2.0f * most);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      if (e < a.E && !((kept >> (e / size)) & 1)) key[i] = 0;
    }
  }
  // One more than is wanted where choices are checked.
  const int rounds = a.k + (sizeof(F) == 4 && !ranked_by_logit ? 1 : 0);
  int mine = -1;
  for (int j = 0; j < rounds; ++j) {
    Key best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = key[i] > best ? key[i] : best;
    const Key top = wave_max(best);
    if (top == 0) break;
    const int from = __builtin_ctzll(__ballot(best == top));
    int slot = 0;
#pragma unroll
    for (int i = V - 1; i > 0; --i) slot = key[i] == top ? i : slot;
    if (key[0] == top) slot = 0;
    const int chosen = from * V + __builtin_amdgcn_readlane(slot, from);
    if (lane == j) mine = chosen;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane * V + i == chosen) key[i] = 0;
  }
  *id = mine;
  return close;
}

template <int DT, int V>
__global__ void __launch_bounds__(kWaves * 64)
topk_kernel(const typename Element<DT>::type *__restrict__ logits, const float *__restrict__ bias, int *__restrict__ ids,
            float *__restrict__ weights, int64_t T, TopkArgs a) {
  __shared__ double buffers[kWaves][64 * V];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
  if (t >= T) return;
  const typename Element<DT>::type *row = logits + t * a.E;
  float logit[V];
  load_logits<DT, V>(row, a.E, lane, logit);
  int id;
  bool again = choose<float, V>(logit, bias, a, lane, reinterpret_cast<float *>(buffers[wave]), &id);

  bool nan = false;  // among all logits
#pragma unroll
  for (int i = 0; i < V; ++i) nan |= logit[i] != logit[i];
  nan = __ballot(nan) != 0;
  float top_logit = kNegInf, sum = 1.0f;  // of all experts
  if (a.score == GEMVTILE_SCORE_SOFTMAX && (!a.norm || bias != nullptr)) {
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) m = logit[i] > m ? logit[i] : m;
    top_logit = wave_max_logit(m);
    float part = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) part += logit[i] == kNegInf ? 0.0f : expf(logit[i] - top_logit);
    sum = wave_sum(part);
  }
  if (bias != nullptr) {
    // Lane j has the j-th choice, lane k the next one.
    const float l = id >= 0 ? widen_logit<DT>(row[id]) : kNegInf;
    const float b = id >= 0 ? bias[id] : 0.0f;
    const bool softmax = a.score == GEMVTILE_SCORE_SOFTMAX;
    const float score = softmax ? (l == kNegInf ? 0.0f : expf(l - top_logit) / sum) : sigmoid(l);
    const float choice = score + b;
    const float next_choice = __shfl_down(choice, 1), next_l = __shfl_down(l, 1), next_b = __shfl_down(b, 1);
    const int next_id = __shfl_down(id, 1);
    // Equal logits with equal biases are a tie in any arithmetic.
    const bool tie = l == next_l && b == next_b;
    const float margin = choice_margin(softmax ? 1.0f / sum : 1.0f, choice, next_choice);
    again |= __ballot(lane < a.k && next_id >= 0 && !tie && !(choice - next_choice > margin)) != 0;
  }
  if (again) choose<double, V>(logit, bias, a, lane, buffers[wave], &id);

  const bool has = lane < a.k;
  const float own = has ? widen_logit<DT>(row[id]) : kNegInf;
  float w;
  if (a.norm) {
    // exp(own - ref) is the score times a number that all of them share; with a
    // sigmoid's 1 + exp(own) below, ref is 0 once a logit is above.
    float ref = wave_max_logit(own);
    if (a.score == GEMVTILE_SCORE_SIGMOID) nan = __ballot(has && own != own) != 0;
    if (a.score == GEMVTILE_SCORE_SOFTMAX) {
      w = ref == kNegInf ? 0.0f : expf(own - ref);
    } else {
      ref = ref < 0.0f ? ref : 0.0f;
      w = own > 0.0f ? 1.0f / (1.0f + expf(-own)) : ref == kNegInf ? 0.0f : expf(own - ref) / (1.0f + expf(own));
    }
    if (!has) w = 0.0f;
    const float total = wave_add(w);
    w = nan ? __builtin_nanf("") : total > 0.0f ? w / total : total;
  } else {
    w = a.score == GEMVTILE_SCORE_SOFTMAX ? (own == kNegInf && !nan ? 0.0f : expf(own - top_logit) / sum) : sigmoid(own);
  }
  if (has) {
    ids[t * a.k + lane] = id;
    weights[t * a.k + lane] = a.scale * w;
  }
}

// ---- gradient ------------------------------------------------------------------
// With g_j = scale * dweight_j, and c_j the chosen scores:
//   softmax               dlogit_e = p_e (g_e - sum_j g_j p_j), g_e = 0 for the others
//   softmax, normalised   dlogit_j = w_j (g_j - sum_i g_i w_i), w the softmax of the chosen logits
//   sigmoid               dlogit_j = g_j c_j (1 - c_j)
//   sigmoid, normalised   the same with (g_j - sum_i g_i w_i) / sum_i c_i for g_j, w = c / sum c
// and 0 for experts not chosen.  Ids outside 0 .. E - 1 are left out.
template <int DT, int V>
__global__ void __launch_bounds__(kWaves * 64)
topk_grad_kernel(const typename Element<DT>::type *__restrict__ logits, const int *__restrict__ ids,
                 const float *__restrict__ dweights, typename Element<DT>::type *__restrict__ dlogits, int64_t T, TopkArgs a) {
  typedef typename Element<DT>::type E_t;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
  if (t >= T) return;
  const E_t *row = logits + t * a.E;
  int id = lane < a.k ? ids[t * a.k + lane] : -1;
  const bool has = id >= 0 && id < a.E;
  if (!has) id = -1;
  const float g = has ? a.scale * dweights[t * a.k + lane] : 0.0f;
  const float own = has ? widen_logit<DT>(row[id]) : kNegInf;
  const bool dense = a.score == GEMVTILE_SCORE_SOFTMAX && !a.norm;
  float p[V];
  float value, dot = 0.0f;  // of the chosen expert; what every expert's score is multiplied with
  if (dense) {
    float logit[V];
    load_logits<DT, V>(row, a.E, lane, logit);
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) m = logit[i] > m ? logit[i] : m;
    m = wave_max_logit(m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = logit[i] == kNegInf ? 0.0f : expf(logit[i] - m);
      sum += p[i];
    }
    sum = wave_add(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] *= inv;
    const float pj = own == kNegInf ? 0.0f : expf(own - m) * inv;
    dot = wave_add(has ? g * pj : 0.0f);
    value = g;
  } else {
    float u, slope;  // score over what all share, and d score / d logit over the same
    const float top = wave_max_logit(own);
    float ref = top;
    if (a.score == GEMVTILE_SCORE_SOFTMAX) {
      u = ref == kNegInf ? 0.0f : expf(own - ref);
      slope = u;
    } else {
      ref = a.norm && ref < 0.0f ? ref : 0.0f;
      const float down = own > 0.0f ? 1.0f / (1.0f + expf(-own)) : ref == kNegInf ? 0.0f : expf(own - ref) / (1.0f + expf(own));
      u = down;
      slope = own > 0.0f ? down * (expf(-own) / (1.0f + expf(-own))) : down / (1.0f + expf(own));
    }
    if (!has) u = slope = 0.0f;
    if (a.norm) {
      const float total = wave_add(u);
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
      const float mean = wave_add(has ? g * u : 0.0f) * inv;
      value = (g - mean) * (slope * inv);
    } else {
      value = g * slope;
    }
  }
  // To the lanes that have the experts.
  float out[V];
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const float v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, value), j));
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane * V + i == e) out[i] += v;
  }
  if (dense) {
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = p[i] * (out[i] - dot);
  }
  E_t *dst = dlogits + t * a.E;
  const int e0 = lane * V;
  if (a.E % V == 0) {
    if (e0 < a.E) {
      E_t v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = round_logit<DT>(out[i]);
      __builtin_memcpy(__builtin_assume_aligned(dst + e0, V * sizeof(E_t) < 16 ? V * sizeof(E_t) : 16), v, sizeof(v));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < a.E) dst[e0 + i] = round_logit<DT>(out[i]);
  }
}

// ---- sorting the slots -----------------------------------------------------------
// A counting sort: slots (t, j) in order, stable, by expert.  Each wave has a run
// of slots and counts its experts in LDS; a slot's row is where its expert begins,
// plus the expert's slots in earlier workgroups, in earlier waves and in earlier
// steps of this wave, plus those of lower lanes (lanes with the same expert find
// one another through a ballot for each bit of the number).  No atomic decides an
// order, so rows never depend on timing.
constexpr int kSortWaves = 8;
constexpr int kSortThreads = kSortWaves * 64;
constexpr int kSortExperts = 1024;

struct SortRun {
  int64_t begin, end;
};
// The slots of a workgroup, and of one of its waves: runs of whole steps of 64.
__device__ inline SortRun sort_run(int64_t begin, int64_t end, int part, int parts) {
  const int64_t steps = (end - begin + 63) / 64;
  int64_t b = begin + steps * part / parts * 64, e = begin + steps * (part + 1) / parts * 64;
  if (e > end) e = end;
  if (b > e) b = e;
  return {b, e};
}

__device__ inline void count_run(const int *ids, SortRun r, int E, uint32_t *count, int lane) {
  for (int64_t i = r.begin + lane; i < r.end; i += 64) {
    const int e = ids[i];
    if (e >= 0 && e < E) atomicAdd(&count[e], 1u);  // a count: its order does not matter
  }
}

// hist [blocks, E]: each workgroup's slots by expert.
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const int *__restrict__ ids, int *__restrict__ hist, int64_t n, int E) {
  __shared__ uint32_t count[kSortExperts];
  for (int e = threadIdx.x; e < E; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const SortRun all = sort_run(0, n, blockIdx.x, gridDim.x);
  count_run(ids, sort_run(all.begin, all.end, threadIdx.x >> 6, kSortWaves), E, count, threadIdx.x & 63);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) hist[static_cast<int64_t>(blockIdx.x) * E + e] = static_cast<int>(count[e]);
}

// hist is NULL for a launch of one workgroup.
__global__ void __launch_bounds__(kSortThreads)
sort_place_kernel(const int *__restrict__ ids, const int *__restrict__ hist, int *__restrict__ offsets, int *__restrict__ pos,
                  int64_t n, int E, int bits) {
  __shared__ uint32_t count[kSortWaves][kSortExperts];  // first a wave's slots by expert, then its next row of each
  __shared__ uint32_t wave_total[kSortWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int e = lane; e < E; e += 64) count[wave][e] = 0;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const SortRun all = sort_run(0, n, blockIdx.x, gridDim.x);
  const SortRun mine = sort_run(all.begin, all.end, wave, kSortWaves);
  count_run(ids, mine, E, count[wave], lane);
  __syncthreads();
  // Thread i has experts 2 i and 2 i + 1: slots ahead in earlier workgroups, and in all.
  uint32_t before[2] = {0, 0}, total[2] = {0, 0};
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int e = 2 * static_cast<int>(threadIdx.x) + s;
    if (e < E) {
      if (hist == nullptr) {
        for (int w = 0; w < kSortWaves; ++w) total[s] += count[w][e];
      } else {
        const int blocks = static_cast<int>(gridDim.x);
#pragma unroll 8
        for (int b = 0; b < blocks; ++b) {
          const uint32_t c = static_cast<uint32_t>(hist[static_cast<int64_t>(b) * E + e]);
          before[s] += b < static_cast<int>(blockIdx.x) ? c : 0u;
          total[s] += c;
        }
      }
    }
  }
  // Exclusive sum of the totals over the workgroup.
  uint32_t scan = total[0] + total[1];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(scan, d);
    if (lane >= d) scan += o;
  }
  if (lane == 63) wave_total[wave] = scan;
  __syncthreads();
  uint32_t start = scan - total[0] - total[1];
  for (int w = 0; w < wave; ++w) start += wave_total[w];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int e = 2 * static_cast<int>(threadIdx.x) + s;
    if (e < E) {
      if (blockIdx.x == 0) {
        offsets[e] = static_cast<int>(start);
        if (e == E - 1) offsets[E] = static_cast<int>(start + total[s]);
      }
      uint32_t next = start + before[s];
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = count[w][e];
        count[w][e] = next;
        next += c;
      }
    }
    start += total[s];
  }
  __syncthreads();
  volatile uint32_t *next_row = count[wave];
  for (int64_t base = mine.begin; base < mine.end; base += 64) {
    const int64_t i = base + lane;
    const bool in = i < mine.end;
    const int e = in ? ids[i] : -1;
    const bool valid = e >= 0 && e < E;
    uint64_t same = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
      const bool one = (e >> b) & 1;
      const uint64_t ones = __ballot(one);
      same &= one ? ones : ~ones;
    }
    const int rank = __builtin_popcountll(same & ((uint64_t{1} << lane) - 1));
    uint32_t row = 0;
    if (valid) row = next_row[e] + static_cast<uint32_t>(rank);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (valid && rank == 0) next_row[e] = row + static_cast<uint32_t>(__builtin_popcountll(same));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (in) pos[i] = valid ? static_cast<int>(row) : -1;
  }
}

template <int DT, int V>
hipError_t launch_topk_v(const void *logits, const float *bias, int *ids, float *weights, int64_t T, const TopkArgs &a,
                         hipStream_t stream) {
  hipLaunchKernelGGL((topk_kernel<DT, V>), dim3(static_cast<unsigned>((T + kWaves - 1) / kWaves)), dim3(kWaves * 64), 0, stream,
                     static_cast<const typename Element<DT>::type *>(logits), bias, ids, weights, T, a);
  return hipGetLastError();
}
template <int DT>
hipError_t launch_topk_dt(const void *logits, const float *bias, int *ids, float *weights, int64_t T, const TopkArgs &a,
                          hipStream_t stream) {
  if (a.E <= 64) return launch_topk_v<DT, 1>(logits, bias, ids, weights, T, a, stream);
  if (a.E <= 128) return launch_topk_v<DT, 2>(logits, bias, ids, weights, T, a, stream);
  if (a.E <= 256) return launch_topk_v<DT, 4>(logits, bias, ids, weights, T, a, stream);
  if (a.E <= 512) return launch_topk_v<DT, 8>(logits, bias, ids, weights, T, a, stream);
  return launch_topk_v<DT, 16>(logits, bias, ids, weights, T, a, stream);
}
template <int DT, int V>
hipError_t launch_topk_grad_v(const void *logits, const int *ids, const float *dweights, void *dlogits, int64_t T,
                              const TopkArgs &a, hipStream_t stream) {
  typedef typename Element<DT>::type E_t;
  hipLaunchKernelGGL((topk_grad_kernel<DT, V>), dim3(static_cast<unsigned>((T + kWaves - 1) / kWaves)), dim3(kWaves * 64), 0,
                     stream, static_cast<const E_t *>(logits), ids, dweights, static_cast<E_t *>(dlogits), T, a);
  return hipGetLastError();
}
template <int DT>
hipError_t launch_topk_grad_dt(const void *logits, const int *ids, const float *dweights, void *dlogits, int64_t T,
                               const TopkArgs &a, hipStream_t stream) {
  if (a.E <= 64) return launch_topk_grad_v<DT, 1>(logits, ids, dweights, dlogits, T, a, stream);
  if (a.E <= 128) return launch_topk_grad_v<DT, 2>(logits, ids, dweights, dlogits, T, a, stream);
  if (a.E <= 256) return launch_topk_grad_v<DT, 4>(logits, ids, dweights, dlogits, T, a, stream);
  if (a.E <= 512) return launch_topk_grad_v<DT, 8>(logits, ids, dweights, dlogits, T, a, stream);
  return launch_topk_grad_v<DT, 16>(logits, ids, dweights, dlogits, T, a, stream);
}

}  // namespace

hipError_t launch_route_topk(int dtype, const void *logits, const float *bias, int *ids, float *weights, const RouteArgs &r,
                             hipStream_t stream) {
  const TopkArgs a = {r.E, r.k, r.groups, r.top_groups, r.group_best, r.score, r.norm, r.scale};
  if (dtype == kF16) return launch_topk_dt<kF16>(logits, bias, ids, weights, r.T, a, stream);
  if (dtype == kBF16) return launch_topk_dt<kBF16>(logits, bias, ids, weights, r.T, a, stream);
  return launch_topk_dt<kF32>(logits, bias, ids, weights, r.T, a, stream);
}

hipError_t launch_route_topk_grad(int dtype, const void *logits, const int *ids, const float *dweights, void *dlogits,
                                  const RouteArgs &r, hipStream_t stream) {
  const TopkArgs a = {r.E, r.k, 1, 1, 1, r.score, r.norm, r.scale};
  if (dtype == kF16) return launch_topk_grad_dt<kF16>(logits, ids, dweights, dlogits, r.T, a, stream);
  if (dtype == kBF16) return launch_topk_grad_dt<kBF16>(logits, ids, dweights, dlogits, r.T, a, stream);
  return launch_topk_grad_dt<kF32>(logits, ids, dweights, dlogits, r.T, a, stream);
}

int route_sort_blocks(int64_t slots) {
  if (slots <= 4096) return 1;
  const int64_t b = (slots + 2047) / 2048;
  return static_cast<int>(b < 64 ? b : 64);
}

hipError_t launch_route_sort(const int *ids, int *offsets, int *pos, int *hist, int64_t slots, int E, hipStream_t stream) {
  const int blocks = route_sort_blocks(slots);
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  if (blocks > 1) {
    hipLaunchKernelGGL(sort_count_kernel, dim3(blocks), dim3(kSortThreads), 0, stream, ids, hist, slots, E);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(sort_place_kernel, dim3(blocks), dim3(kSortThreads), 0, stream, ids, blocks > 1 ? hist : nullptr, offsets,
                     pos, slots, E, bits);
  return hipGetLastError();
}

}  // namespace gt
