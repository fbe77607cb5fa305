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
// 16 lanes have one token (64 lanes where there are more than 256 experts or 14
// choices), each V experts that follow one another.  An expert's key is its choice,
// rounded down to 31 bits less those of its number, and the number, inverted: keys
// are all different and tied choices are in order.  A round of the choice is then
// the largest key below the last one, one subtraction and half a maximum an expert
// and a maximum over the lanes through DPP; nothing is marked as taken, and the
// key says whose it is.
//
// Bound by vector instructions, 280 a token of 256 experts, half of them in the rounds,
// which pass over all of a lane's numbers, dropped groups' too (16384 tokens, 8 of 256 of
// bf16 logits: 6.7 us, with a sigmoid and a bias 10.7, in 4 of 8 groups 12.1; with a
// wave a token, as at 16 of 256, 13.2, 19.3 and 22.1).
//
// Ids are those of exact arithmetic.  16-bit logits fit a key as they are.  Scores,
// and logits of 32 bits, are rounded; each decision (a choice against the next, the
// last kept group against the first dropped) is checked afterwards against the
// rounding and against what FP32 scores can be off.  Of a closer decision, one in some
// hundred tokens, the few numbers that it is about are worked out in FP64, and where
// that does not settle it the token is done again in FP64 by the whole wave.
#include "device_common.hpp"
#include "../../include/gemvtile.h"
#include "kernels.hpp"
#include "wave_ops.hpp"

namespace gt {

namespace {

constexpr int kWaves = 4;  // of a workgroup
constexpr float kNegInf = -__builtin_inff();

// What FP32 scores can be off, u = 2^-24.  fast_exp(v) of either sign is off by
// (1.25 |v| + 2) u of itself: the product with log2(e), that number's own rounding, and the
// instruction's unit in the last place.
//
// Sigmoid: s (1 - s) (1.25 |v| + 2) <= 0.7 u, its sum and reciprocal 3 u more: 4 u.
//
// Softmax, v = logit - largest, rounded: an exponential is off by (2.25 |v| + 2) u of itself,
// at most 2.1 u of the largest one.  Their sum over E <= 1024 is off by what they are off in
// the mean, (2.25 * 4.44 + 2) u (the mean of |v| is largest, 4.44, with one logit on top and
// 1023 of them 5.44 below), and by 10 u for a tree of 4 + 6 levels: with its reciprocal 23 u.
// That factor is all scores' alike, so of the difference of two it is 23 u of the difference,
// which is at most the largest score p; with the exponentials and their products, 3.1 u of p
// each, two scores' difference is off by at most 30 u of p, two sums of two by 59 u.  Twice
// score_error, 32 u of p, is in the margin of two choices; twice that, 64 u, in that of two
// groups.
//
// Adding a bias rounds by u of the choice.  A choice x that is far below in FP32 cannot be
// ahead of c in truth, however large it is: it would take |x| within 2^-22 of |c|.
__device__ inline float score_error(bool softmax, float top_score) { return softmax ? 0x1p-20f * top_score : 0x1p-22f; }
// How far apart two choices have to be; `step` is that of the keys.
__device__ inline float choice_margin(float score_error, float a, float b, float step) {
  return 2.0f * score_error + 0x1p-23f * (__builtin_fabsf(a) + __builtin_fabsf(b)) + step;
}
// What a group's one or two best can be off, and their sum.
__device__ inline float group_error(float score_error, float first, float second) {
  return 2.0f * score_error + 0x1p-23f * (__builtin_fabsf(first) + __builtin_fabsf(second));
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
__device__ inline uint64_t wave_max(uint64_t v) {  // the upper halves, then the lower ones of those that have it
  const uint32_t high = static_cast<uint32_t>(v >> 32), top = wave_max(high);
  return static_cast<uint64_t>(top) << 32 | wave_max(high == top ? static_cast<uint32_t>(v) : 0u);
}
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

// The lane's V biases, -inf behind the last expert.
template <int V>
__device__ inline void load_bias(const float *bias, int E, int lane, float *out) {
  const int e0 = lane * V;
  if (V % 4 == 0 && E % V == 0 && (reinterpret_cast<uintptr_t>(bias) & 15) == 0) {
    if (e0 < E) {
      __builtin_memcpy(out, __builtin_assume_aligned(bias + e0, V % 4 == 0 ? 16 : 4), V * sizeof(float));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) out[i] = kNegInf;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = e0 + i < E ? bias[e0 + i] : kNegInf;
  }
}

__device__ inline float sigmoid(float v) {
  const float e = expf(v < 0 ? v : -v);
  return (v < 0 ? e : 1.0f) / (1.0f + e);
}
__device__ inline double sigmoid(double v) {
  const double e = exp(v < 0 ? v : -v);
  return (v < 0 ? e : 1.0) / (1.0 + e);
}

struct TopkArgs {
  int E, k, groups, top_groups, group_best, score, norm;
  float scale;
};

// ---- the choice in FP64 --------------------------------------------------------
// By a whole wave for one token: lane j < k gets the id of the j-th choice.  `buf`
// holds E numbers of the wave's own, choices (their bits) and then keys.  Few tokens come
// here, so the code is never in the instruction cache and its length is what it costs:
// loops, nothing unrolled.
template <int DT>
__device__ __attribute__((always_inline)) inline int choose_exactly(const typename Element<DT>::type *row, const float *bias, TopkArgs a,
                                                        uint64_t *buf) {
  typedef KeyOf<double> Keys;
  const auto put = [&](int e, double v) { buf[e] = __builtin_bit_cast(uint64_t, v); };
  const auto get = [&](int e) { return __builtin_bit_cast(double, buf[e]); };
  // What the wave read of this memory before (another token's keys, numbers in FP32) has
  // been read.
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const int lane = threadIdx.x & 63;
  const bool softmax = a.score == GEMVTILE_SCORE_SOFTMAX;
  const int size = a.E / a.groups;
  const bool sums = a.groups > 1 && a.group_best == 2 && size > 1;
  const bool scored = bias != nullptr || sums;
  float m = 0.0f;
  double inv = 1;
  if (scored && softmax) {
    m = kNegInf;
#pragma clang loop unroll(disable)
    for (int e = lane; e < a.E; e += 64) {
      const float l = widen_logit<DT>(row[e]);
      m = l > m ? l : m;
    }
    m = wave_max_logit(m);
  }
  // A softmax's exponentials, or a sigmoid.
  double sum = 0;
#pragma clang loop unroll(disable)
  for (int e = lane; e < a.E; e += 64) {
    const double l = static_cast<double>(widen_logit<DT>(row[e]));
    double v = l;
    if (scored) {
      const double x = softmax ? l - static_cast<double>(m) : l < 0 ? l : -l;
      const double p = softmax && l == kNegInf ? 0 : exp(x);
      sum += p;
      v = softmax ? p : (l < 0 ? p : 1) / (1 + p);
    }
    put(e, v);
  }
  if (scored && softmax) {
    sum = wave_add(sum);
    inv = sum == 0 ? 1 : sum;  // 0: every logit is -inf
  }
#pragma clang loop unroll(disable)
  for (int e = lane; e < a.E; e += 64)
    if (scored) put(e, get(e) / inv + (bias != nullptr ? static_cast<double>(bias[e]) : 0.0));
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  uint64_t kept = 1;
  if (a.groups > 1) {
    // Lane g works out group g.
    uint64_t gkey = 0;
    if (lane < a.groups) {
      double first = get(lane * size), second = 0;
      uint64_t k1 = Keys::of(first), k2 = 0;
#pragma unroll 4
      for (int i = 1; i < size; ++i) {
        const double v = get(lane * size + i);
        const uint64_t kv = Keys::of(v);
        const bool ahead = kv > k1, next = kv > k2;
        second = ahead ? first : next ? v : second;
        k2 = ahead ? k1 : next ? kv : k2;
        first = ahead ? v : first;
        k1 = ahead ? kv : k1;
      }
      gkey = Keys::of(sums ? first + second : first);
    }
    int rank = 0;  // groups ahead of this one
#pragma clang loop unroll(disable)
    for (int o = 0; o < a.groups; ++o) {
      const uint64_t other =
          static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(gkey >> 32), o))) << 32 |
          static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(gkey), o));
      rank += other > gkey || (other == gkey && o < lane) ? 1 : 0;
    }
    kept = __ballot(lane < a.groups && rank < a.top_groups);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  // Each lane has a run of experts; buf holds their keys from here on.
  const int run = (a.E + 63) / 64, e0 = lane * run;
  uint64_t best = 0;
  int at = 0;
#pragma clang loop unroll(disable)
  for (int e = e0; e < e0 + run && e < a.E; ++e) {
    const uint64_t key = (kept >> (e / size)) & 1 ? Keys::of(bias != nullptr ? get(e) : static_cast<double>(widen_logit<DT>(row[e]))) : 0;
    buf[e] = key;
    at = key > best ? e : at;
    best = key > best ? key : best;
  }
  int mine = -1;
#pragma clang loop unroll(disable)
  for (int j = 0; j < a.k; ++j) {
    const uint64_t top = wave_max(best);
    const int from = __builtin_ctzll(__ballot(best == top));  // the lowest lane, and in it the lowest expert
    const int chosen = __builtin_amdgcn_readlane(at, from);
    if (lane == j) mine = chosen;
    if (lane == from) {
      buf[chosen] = 0;
      best = 0;
#pragma clang loop unroll(disable)
      for (int e = e0; e < e0 + run && e < a.E; ++e) {
        const uint64_t key = buf[e];
        at = key > best ? e : at;
        best = key > best ? key : best;
      }
    }
  }
  return mine;
}

// ---- the choice in FP32 ----------------------------------------------------------
// Over the L lanes of a token, in all of them.
template <int L>
__device__ inline uint32_t part_max(uint32_t v) {
  if constexpr (L == 16) return max_of_16_lanes(v);
  else return wave_max(v);
}
// NaN left aside; -inf of nothing.
template <int L>
__device__ inline float part_max(float v) {
  return KeyOf<float>::value(part_max<L>(KeyOf<float>::of(v == v ? v : kNegInf)));
}
// Whether it is so in any of the token's lanes.
template <int L>
__device__ inline bool part_any(bool v, int lane) {
  const uint64_t b = __ballot(v);
  if constexpr (L == 64) return b != 0;
  return ((b >> (lane & 48)) & 0xffffu) != 0;
}
// e^v by the hardware's power of two; what it is off stands at score_error.
__device__ inline float fast_exp(float v) { return __builtin_amdgcn_exp2f(v * 0x1.715476p+0f); }
__device__ inline float fast_sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + fast_exp(-v)); }

template <int N>
__device__ inline float tree_sum(const float *v) {
  if constexpr (N == 1) return v[0];
  else return tree_sum<N / 2>(v) + tree_sum<N / 2>(v + N / 2);
}

template <int CTRL>
__device__ inline float dpp_move(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
// A group's two best from those of two of its parts.
struct Best {
  float first, second;
};
__device__ inline Best merge(Best a, float first, float second) {
  return {__builtin_fmaxf(a.first, first),
          __builtin_fmaxf(__builtin_fminf(a.first, first), __builtin_fmaxf(a.second, second))};
}
__device__ inline Best merge(Best a, float v) {
  return {__builtin_fmaxf(a.first, v), __builtin_amdgcn_fmed3f(a.first, a.second, v)};
}

constexpr int kMaxGroups = 64;
template <int L, int V>
union TopkShared {
  uint64_t exact[L * V];  // of one token
  struct {
    float value[64 / L][L * V];
    float group[64 / L][kMaxGroups], error[64 / L][kMaxGroups];
  } fast;
};

template <int DT, int L, int V>
__global__ void __launch_bounds__(kWaves * 64)
topk_kernel(const typename Element<DT>::type *__restrict__ logits, const float *__restrict__ bias, int *__restrict__ ids,
            float *__restrict__ weights, int64_t T, TopkArgs a) {
  constexpr int kTokens = 64 / L;  // of a wave
  constexpr int kIndexBits = __builtin_ctz(L * V);
  __shared__ TopkShared<L, V> shared[kWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = lane / L, sub = lane & (L - 1);
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kTokens;
  if (t0 >= T) return;  // the whole wave
  const bool there = t0 + part < T;
  const int64_t t = there ? t0 + part : T - 1;  // lanes without a token do the last one's work
  const typename Element<DT>::type *row = logits + t * a.E;
  const bool biased = bias != nullptr;
  const bool softmax = a.score == GEMVTILE_SCORE_SOFTMAX;
  const int size = a.E / a.groups;
  const bool sums = a.groups > 1 && a.group_best == 2 && size > 1;
  const bool rounded = biased || DT == kF32;  // what the keys hold is not exact

  float logit[V], value[V];
  load_logits<DT, V>(row, a.E, sub, logit);
  float top_logit = kNegInf, sum = 1.0f;  // of all experts
  const bool scored = biased || sums;
  if (softmax && (scored || !a.norm)) {
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) m = logit[i] > m ? logit[i] : m;
    top_logit = part_max<L>(m);
#pragma unroll
    for (int i = 0; i < V; ++i) value[i] = logit[i] == kNegInf ? 0.0f : fast_exp(logit[i] - top_logit);
    sum = lanes_sum<L>(tree_sum<V>(value));
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < V; ++i) value[i] *= inv;
  } else if (scored) {
#pragma unroll
    for (int i = 0; i < V; ++i) value[i] = fast_sigmoid(logit[i]);
  }
  const float wrong = score_error(softmax, 1.0f / sum);
  float own_bias[V];
  if (biased) {
    load_bias<V>(bias, a.E, sub, own_bias);
#pragma unroll
    for (int i = 0; i < V; ++i) value[i] += own_bias[i];
  } else if (!sums) {
#pragma unroll
    for (int i = 0; i < V; ++i) value[i] = logit[i];
  }
  // A choice that is NaN (its logit or its bias is, or the softmax) is left to FP64.
  bool nan = false;
#pragma unroll
  for (int i = 0; i < V; ++i) nan |= biased ? value[i] != value[i] : logit[i] != logit[i];
  nan = part_any<L>(nan, lane);
  bool again = nan && (scored || rounded || a.groups > 1);
  if (biased && nan) {  // all lanes of the token; from here on it is about the logits
    nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) nan |= logit[i] != logit[i];
    nan = part_any<L>(nan, lane);
  }
  // A softmax beside an infinite logit is NaN, whatever is chosen.  (Where the largest logit
  // is not known, it is among the chosen ones.)
  nan |= top_logit == __builtin_inff();

  // ---- groups: value[] is what they count by
  uint32_t dropped = 0;  // experts of this lane (as bits) in groups that are not kept
  if (a.groups > 1) {
    bool close = false;
    const int lanes = size / V;  // of a group, if that is a power of two
    if (lanes * V == size && (lanes & (lanes - 1)) == 0) {
      Best b = {kNegInf, kNegInf};
#pragma unroll
      for (int i = 0; i < V; ++i) b = merge(b, value[i]);  // with a NaN the token is done again
      if (lanes >= 2) b = merge(b, dpp_move<0xB1>(b.first), dpp_move<0xB1>(b.second));
      if (lanes >= 4) b = merge(b, dpp_move<0x4E>(b.first), dpp_move<0x4E>(b.second));
      if (lanes >= 8) b = merge(b, dpp_move<0x141>(b.first), dpp_move<0x141>(b.second));
      if (lanes >= 16) b = merge(b, dpp_move<0x140>(b.first), dpp_move<0x140>(b.second));
      if (lanes >= 32) b = merge(b, __shfl_xor(b.first, 16), __shfl_xor(b.second, 16));
      const int mine = sub / lanes;
      const bool real = mine < a.groups;
      const float counts = sums ? b.first + b.second : b.first;
      again |= part_any<L>(counts != counts, lane);
      int rank = 0;  // groups ahead of this one
      for (int o = 0; o < a.groups; ++o) {
        const float other = __shfl(counts, part * L + o * lanes);
        rank += other > counts || (other == counts && o < mine) ? 1 : 0;
      }
      const bool kept = real && rank < a.top_groups;
      if (!kept) dropped = ~0u;
      if (scored && a.top_groups < a.groups) {
        // The last kept group against the first dropped one, and the largest error of any.
        const float low = -part_max<L>(kept ? -counts : kNegInf), high = part_max<L>(real && !kept ? counts : kNegInf);
        const float error = real ? group_error(wrong, b.first, sums ? b.second : 0.0f) : 0.0f;
        const float most = __builtin_bit_cast(float, part_max<L>(__builtin_bit_cast(uint32_t, error)));
        close = !(low - high > 2.0f * most);
        if (__ballot(close) != 0 && !softmax) {
          // In FP64, by the choices that count alone.  Where others come near them,
          // the group counts by more than these.
          const int need = sums ? 2 : 1;
          const float least = sums ? b.second : b.first;
          const float edge = least - choice_margin(wrong, least, least, 0.0f);
          int count = 0;
          float l1 = 0.0f, b1 = 0.0f, l2 = 0.0f, b2 = 0.0f;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (sub * V + i < a.E && value[i] >= edge) {
              l2 = l1;
              b2 = b1;
              l1 = logit[i];
              b1 = biased ? own_bias[i] : 0.0f;
              ++count;
            }
          }
          double exact = count > 0 ? sigmoid(static_cast<double>(l1)) + static_cast<double>(b1) : 0.0;
          if (count > 1) exact += sigmoid(static_cast<double>(l2)) + static_cast<double>(b2);
          for (int d = 1; d < lanes; d <<= 1) {
            exact += __shfl_xor(exact, d);
            count += __shfl_xor(count, d);
          }
          const bool unclear = part_any<L>(real && count != need, lane);
          rank = 0;
          for (int o = 0; o < a.groups; ++o) {
            const double other = __shfl(exact, part * L + o * lanes);
            rank += other > exact || (other == exact && o < mine) ? 1 : 0;
          }
          if (close && !unclear) {
            dropped = real && rank < a.top_groups ? 0 : ~0u;
            close = false;
          }
        }
      }
    } else {
      auto &s = shared[wave].fast;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (sub * V + i < a.E) s.value[part][sub * V + i] = value[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      for (int o = sub; o < a.groups; o += L) {
        Best b = {kNegInf, kNegInf};
        for (int i = 0; i < size; ++i) b = merge(b, s.value[part][o * size + i]);
        s.group[part][o] = sums ? b.first + b.second : b.first;
        s.error[part][o] = group_error(wrong, b.first, sums ? b.second : 0.0f);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      float low = __builtin_inff(), high = kNegInf, most = 0.0f;
      bool none = false;
      for (int o = sub; o < a.groups; o += L) {
        const float counts = s.group[part][o];
        none |= counts != counts;
        int rank = 0;
        for (int p = 0; p < a.groups; ++p) {
          const float other = s.group[part][p];
          rank += other > counts || (other == counts && p < o) ? 1 : 0;
        }
        const bool kept = rank < a.top_groups;
        low = kept ? __builtin_fminf(low, counts) : low;
        high = kept ? high : __builtin_fmaxf(high, counts);
        const float error = s.error[part][o];
        most = error > most || error != error ? error : most;
        s.error[part][o] = kept ? 1.0f : 0.0f;  // only this lane reads the errors of its groups
      }
      again |= part_any<L>(none, lane);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = sub * V + i;
        if (e < a.E && s.error[part][e / size] == 0.0f) dropped |= 1u << i;
      }
      if (scored && a.top_groups < a.groups) {
        low = -part_max<L>(-low);
        high = part_max<L>(high);
        most = __builtin_bit_cast(float, part_max<L>(__builtin_bit_cast(uint32_t, most)));
        close = !(low - high > 2.0f * most);
      }
    }
    again |= close;
  }
  if (!biased && sums) {
#pragma unroll
    for (int i = 0; i < V; ++i) value[i] = logit[i];
  }

  // ---- keys: 1 + the rounded choice above the inverted number; 0: not to be chosen
  uint32_t key[V];
  float step = 0.0f, lowest = kNegInf;  // the keys' step; what the lowest of them reach up to
  if (rounded) {
    // Equal steps over 2 below the largest choice (16 of logits); further down all are
    // alike, and settled as whatever is too near is.
    constexpr uint32_t kSteps = (1u << (31 - kIndexBits < 23 ? 31 - kIndexBits : 23)) - 4;  // FP32 counts them all
    float high = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) high = __builtin_fmaxf(high, value[i]);
    high = part_max<L>(high);
    again |= !(__builtin_fabsf(high) < __builtin_inff());
    const float range = biased ? 2.0f : 16.0f, scale = static_cast<float>(kSteps) / range;
    const float base = 1.0f - (high - range) * scale;
    step = 2.0f * range / static_cast<float>(kSteps);
    lowest = high - range + step;
#pragma unroll
    for (int i = 0; i < V; ++i)
      key[i] = static_cast<uint32_t>(
          __builtin_amdgcn_fmed3f(__builtin_fmaf(value[i], scale, base), 1.0f, static_cast<float>(kSteps + 1)));
  } else {
    // All bits that differ among 16-bit numbers.
    constexpr int kShift = DT == kBF16 ? 16 : 13;
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = (KeyOf<float>::of(value[i]) >> kShift) + 1;
  }
  {
    // Bits of the lane's experts that can be chosen.
    const int count = a.E - sub * V < 0 ? 0 : a.E - sub * V < V ? a.E - sub * V : V;
    const uint32_t open = ((1u << count) - 1u) & ~dropped;
    const uint32_t number = static_cast<uint32_t>(L * V - V - sub * V);
#pragma unroll
    for (int i = 0; i < V; ++i)
      key[i] = (key[i] << kIndexBits | (number + (V - 1 - i))) & static_cast<uint32_t>(static_cast<int>(open << (31 - i)) >> 31);
  }

  // ---- rounds: lane j gets the j-th largest key, two more than are wanted where keys are rounded
  uint32_t best = key[0];
#pragma unroll
  for (int i = 1; i < V; ++i) best = key[i] > best ? key[i] : best;
  uint32_t mine = 0;
  const int rounds = a.k + (rounded ? 2 : 0);
  for (int j = 0; j < rounds; ++j) {
    const uint32_t top = part_max<L>(best);
    if (sub == j) mine = top;
    // The largest key below: keys less top wrap round to the upper half.
    uint32_t below = key[0] - top;
#pragma unroll
    for (int i = 1; i < V; ++i) below = key[i] - top > below ? key[i] - top : below;
    best = below & 0x80000000u ? below + top : 0;
  }
  const auto number = [](uint32_t key) { return key == 0 ? -1 : L * V - 1 - static_cast<int>(key & (L * V - 1)); };
  int id = number(mine);
  float l = id >= 0 ? widen_logit<DT>(row[id]) : kNegInf;

  if (rounded) {
    // Lane j has the j-th choice, lanes k and k + 1 the next ones.
    const float b = biased && id >= 0 ? bias[id] : 0.0f;
    float choice = l;
    if (biased)
      choice = (softmax ? (l == kNegInf ? 0.0f : fast_exp(l - top_logit) / sum) : fast_sigmoid(l)) + b;
    // What the numbers with this key or a lower one reach up to: the lowest key stands for
    // all further down.
    const float reach = mine >> kIndexBits <= 1 ? __builtin_fmaxf(choice, lowest) : choice;
    const float next_choice = __shfl_down(reach, 1), next_l = __shfl_down(l, 1), next_b = __shfl_down(b, 1);
    const uint32_t next_key = static_cast<uint32_t>(__shfl_down(static_cast<int>(mine), 1));
    const bool judged = sub < a.k && next_key != 0;
    // Equal logits with equal biases are a tie in any arithmetic.
    const bool tie = l == next_l && b == next_b;
    const bool good = tie || (biased ? choice - next_choice > choice_margin(wrong, choice, next_choice, step) : l > next_l);
    const bool bad = part_any<L>(judged && !good, lane);
    // Where the last choice and the next one tie, or share a step, or are too near,
    // others may be as near: not if the one after next is further down.
    const bool edge = sub == a.k - 1 && judged && (tie || !good || mine >> kIndexBits == next_key >> kIndexBits);
    bool alone = true;
    if (__ballot(edge || bad) != 0) {
      const int from = part * L + a.k - 1;
      const float last = __shfl(choice, from), after = __shfl(reach, from + 2);
      const float last_l = __shfl(l, from), last_b = __shfl(b, from);
      const uint32_t last_key = static_cast<uint32_t>(__shfl(static_cast<int>(mine), from));
      const uint32_t after_key = static_cast<uint32_t>(__shfl(static_cast<int>(mine), from + 2));
      alone = after_key == 0 || (last_key >> kIndexBits != after_key >> kIndexBits &&
                                 (!biased || last - after > choice_margin(wrong, last, after, step)));
      const bool asked = __shfl(static_cast<int>(edge), from) != 0 && !alone;
      // Each other one has to be such a tie, or further down.
      bool doubt = false;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (key[i] != 0 && key[i] < last_key) {
          const float other = biased ? value[i] : logit[i];
          const bool same = logit[i] == last_l && (!biased || own_bias[i] == last_b);
          doubt |= !same && !(biased ? last - other > choice_margin(wrong, last, other, step) : last_l > other);
        }
      }
      again |= part_any<L>(doubt && asked, lane);
      again |= bad && (!alone || (biased && softmax));
      if (__ballot(bad && !again) != 0) {
        // The k + 2 in FP64: lane j takes the place that its number has among them.
        const bool in = sub < rounds && id >= 0;
        double exact = static_cast<double>(l);
        if (biased) exact = sigmoid(exact) + static_cast<double>(b);
        int place = 0;
        for (int o = 0; o < rounds; ++o) {
          const double other = __shfl(exact, part * L + o);
          const int other_id = __shfl(id, part * L + o);
          place += other_id >= 0 && (other > exact || (other == exact && other_id < id)) ? 1 : 0;
        }
        const int to = (part * L + (in ? place : sub)) * 4;
        const int new_id = __builtin_amdgcn_ds_permute(to, id);
        const float new_l = __builtin_bit_cast(float, __builtin_amdgcn_ds_permute(to, __builtin_bit_cast(int, l)));
        if (bad) {
          id = new_id;
          l = new_l;
        }
      }
    }
  }
  uint64_t todo = __ballot(again && there);
  while (todo != 0) {
    const int p = __builtin_ctzll(todo) / L;
    todo &= L == 64 ? 0 : ~(uint64_t{0xffff} << (16 * p));
    const int exact = choose_exactly<DT>(logits + (t0 + p) * a.E, bias, a, shared[wave].exact);
    const int moved = __shfl(exact, sub);
    if (part == p) {
      id = moved;
      l = id >= 0 ? widen_logit<DT>(row[id]) : kNegInf;
    }
  }

  const bool has = sub < a.k;
  const float own = has ? l : kNegInf;
  float w;
  if (a.norm) {
    // exp(own - ref) is the score times a number that all of them share; with a
    // sigmoid's 1 + exp(own) below, ref is 0 once a logit is above.
    float ref = part_max<L>(own);
    if (!softmax) nan = part_any<L>(has && own != own, lane);
    if (softmax) {
      w = ref == kNegInf ? 0.0f : expf(own - ref);
    } else {
      ref = ref < 0.0f ? ref : 0.0f;
      w = own > 0.0f ? 1.0f / (1.0f + expf(-own)) : ref == kNegInf ? 0.0f : expf(own - ref) / (1.0f + expf(own));
    }
    if (!has) w = 0.0f;
    const float total = lanes_sum<L>(w);
    w = nan ? __builtin_nanf("") : total > 0.0f ? w / total : total;
  } else {
    w = softmax ? (own == kNegInf && !nan ? 0.0f : expf(own - top_logit) / sum) : sigmoid(own);
  }
  if (has && there) {
    ids[t * a.k + sub] = id;
    weights[t * a.k + sub] = a.scale * w;
  }
}

// ---- gradient ------------------------------------------------------------------
// With g_j = scale * dweight_j, and c_j the chosen scores:
//   softmax               dlogit_e = p_e (g_e - sum_j g_j p_j), g_e = 0 for the others
//   softmax, normalised   dlogit_j = w_j (g_j - sum_i g_i w_i), w the softmax of the chosen logits
//   sigmoid               dlogit_j = g_j c_j (1 - c_j)
//   sigmoid, normalised   the same with (g_j - sum_i g_i w_i) / sum_i c_i for g_j, w = c / sum c
// and 0 for experts not chosen.  Ids outside 0 .. E - 1 are left out.  Rows are written
// whole, by the lanes that have the experts: 8200 tokens, 6 of 128, in 3.9 us, of which
// bytes are 0.9 and the rest a launch and a chain of loads, reductions and stores
// (16384 tokens, 8 of 256 4.6 us, of 512 6.3; without LDS, each lane comparing its
// experts with each of the k, 6.0 and 10.8).
template <int DT, int L, int V>
__global__ void __launch_bounds__(kWaves * 64)
topk_grad_kernel(const typename Element<DT>::type *__restrict__ logits, const int *__restrict__ ids,
                 const float *__restrict__ dweights, typename Element<DT>::type *__restrict__ dlogits, int64_t T, TopkArgs a) {
  typedef typename Element<DT>::type E_t;
  constexpr int kTokens = 64 / L;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = lane / L, sub = lane & (L - 1);
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kTokens;
  if (t0 >= T) return;  // the whole wave
  const bool there = t0 + part < T;
  const int64_t t = there ? t0 + part : T - 1;
  const bool softmax = a.score == GEMVTILE_SCORE_SOFTMAX;
  const bool dense = softmax && !a.norm;
  const E_t *row = logits + t * a.E;
  int id = sub < a.k ? ids[t * a.k + sub] : -1;
  float g = sub < a.k ? a.scale * dweights[t * a.k + sub] : 0.0f;
  float p[V];  // the logits, then their scores
  if (dense) load_logits<DT, V>(row, a.E, sub, p);
  const bool has = id >= 0 && id < a.E;
  if (!has) id = -1;
  if (!has) g = 0.0f;
  const float own = has ? widen_logit<DT>(row[id]) : kNegInf;
  float value, dot = 0.0f;  // of the chosen expert; what every expert's score is multiplied with
  if (dense) {
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) m = p[i] > m ? p[i] : m;
    m = part_max<L>(m);
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = p[i] == kNegInf ? 0.0f : expf(p[i] - m);
    const float sum = lanes_sum<L>(tree_sum<V>(p));
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] *= inv;
    const float pj = own == kNegInf ? 0.0f : expf(own - m) * inv;
    dot = lanes_sum<L>(has ? g * pj : 0.0f);
    value = g;
  } else {
    float u, slope;  // score over what all share, and d score / d logit over the same
    float ref = part_max<L>(own);
    if (softmax) {
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
      const float total = lanes_sum<L>(u);
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
      const float mean = lanes_sum<L>(has ? g * u : 0.0f) * inv;
      value = (g - mean) * (slope * inv);
    } else {
      value = g * slope;
    }
  }
  // To the lanes that have the experts, through LDS: pieces of W experts, those of
  // neighbouring lanes beside one another.
  constexpr int W = V < 4 ? V : 4;
  typedef float Piece __attribute__((ext_vector_type(W)));
  __shared__ __attribute__((aligned(16))) float spread[kWaves][64 / L][L * V];
  float *const mine = spread[wave][part];
#pragma unroll
  for (int i = 0; i < V; i += W) *reinterpret_cast<Piece *>(mine + i * L + sub * W) = Piece(0.0f);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (has) mine[id % V / W * W * L + id / V * W + id % W] = value;  // ids are different
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  float out[V];
#pragma unroll
  for (int i = 0; i < V; i += W) {
    const Piece v = *reinterpret_cast<const Piece *>(mine + i * L + sub * W);
#pragma unroll
    for (int j = 0; j < W; ++j) out[i + j] = v[j];
  }
  if (dense) {
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = p[i] * (out[i] - dot);
  }
  if (!there) return;
  E_t *dst = dlogits + t * a.E;
  const int e0 = sub * V;
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
constexpr int kSortLoads = 16;  // rows of counts that a thread reads together

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

// Four steps' numbers are on their way together, also where there are fewer.
__device__ inline void count_run(const int *ids, SortRun r, int E, uint32_t *count, int lane) {
  for (int64_t base = r.begin; base < r.end; base += 256) {
    int e[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int64_t i = base + s * 64 + lane;
      e[s] = ids[i < r.end ? i : r.end - 1];
      if (i >= r.end) e[s] = -1;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (e[s] >= 0 && e[s] < E) atomicAdd(&count[e[s]], 1u);  // a count: its order does not matter
  }
}

// Threads that share an expert's column of `hist`.
__device__ inline int column_parts(int E) { return E <= 64 ? 8 : E <= 128 ? 4 : E <= 256 ? 2 : 1; }

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
  __shared__ uint32_t ahead[kSortExperts], all_of[kSortExperts];  // an expert's slots in earlier workgroups, and in all
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int e = lane; e < E; e += 64) count[wave][e] = 0;
  for (int e = threadIdx.x; e < E; e += kSortThreads) ahead[e] = all_of[e] = 0;
  __syncthreads();
  if (hist != nullptr) {
    const int parts = column_parts(E), blocks = static_cast<int>(gridDim.x), mine = static_cast<int>(blockIdx.x);
    for (int c = threadIdx.x; c < E * parts; c += kSortThreads) {
      const int part = c / E, e = c - part * E;
      const int past = blocks * (part + 1) / parts;
      uint32_t before = 0, total = 0;
      int b = blocks * part / parts;
      for (; b + kSortLoads <= past; b += kSortLoads) {
#pragma unroll
        for (int i = 0; i < kSortLoads; ++i) {
          const uint32_t v = static_cast<uint32_t>(hist[static_cast<int64_t>(b + i) * E + e]);
          before += b + i < mine ? v : 0u;
          total += v;
        }
      }
      if (b < past) {  // fewer rows, on their way together as well
        uint32_t v[kSortLoads];
#pragma unroll
        for (int i = 0; i < kSortLoads; ++i)
          v[i] = static_cast<uint32_t>(hist[static_cast<int64_t>(b + i < past ? b + i : past - 1) * E + e]);
#pragma unroll
        for (int i = 0; i < kSortLoads; ++i) {
          if (b + i >= past) v[i] = 0;
          before += b + i < mine ? v[i] : 0u;
          total += v[i];
        }
      }
      atomicAdd(&ahead[e], before);  // counts: their order does not matter
      atomicAdd(&all_of[e], total);
    }
  }
  const SortRun all = sort_run(0, n, blockIdx.x, gridDim.x);
  const SortRun mine = sort_run(all.begin, all.end, wave, kSortWaves);
  count_run(ids, mine, E, count[wave], lane);
  __syncthreads();
  // Thread i has experts 2 i and 2 i + 1.
  uint32_t before[2] = {0, 0}, total[2] = {0, 0};
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int e = 2 * static_cast<int>(threadIdx.x) + s;
    if (e < E) {
      before[s] = ahead[e];
      total[s] = all_of[e];
      if (hist == nullptr) {
        for (int w = 0; w < kSortWaves; ++w) total[s] += count[w][e];
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
  int coming = mine.begin + lane < mine.end ? ids[mine.begin + lane] : -1;
  for (int64_t base = mine.begin; base < mine.end; base += 64) {
    const int64_t i = base + lane;
    const bool in = i < mine.end;
    const int e = coming;
    coming = i + 64 < mine.end ? ids[i + 64] : -1;
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

template <int DT, int L, int V>
hipError_t launch_topk_v(const void *logits, const float *bias, int *ids, float *weights, int64_t T, const TopkArgs &a,
                         hipStream_t stream) {
  const int64_t tokens = kWaves * (64 / L);
  hipLaunchKernelGGL((topk_kernel<DT, L, V>), dim3(static_cast<unsigned>((T + tokens - 1) / tokens)), dim3(kWaves * 64), 0,
                     stream, static_cast<const typename Element<DT>::type *>(logits), bias, ids, weights, T, a);
  return hipGetLastError();
}
// 16 lanes hold the k choices and two more.
template <int DT>
hipError_t launch_topk_dt(const void *logits, const float *bias, int *ids, float *weights, int64_t T, const TopkArgs &a,
                          hipStream_t stream) {
  if (a.k <= 14) {
    if (a.E <= 16) return launch_topk_v<DT, 16, 1>(logits, bias, ids, weights, T, a, stream);
    if (a.E <= 32) return launch_topk_v<DT, 16, 2>(logits, bias, ids, weights, T, a, stream);
    if (a.E <= 64) return launch_topk_v<DT, 16, 4>(logits, bias, ids, weights, T, a, stream);
    if (a.E <= 128) return launch_topk_v<DT, 16, 8>(logits, bias, ids, weights, T, a, stream);
    if (a.E <= 256) return launch_topk_v<DT, 16, 16>(logits, bias, ids, weights, T, a, stream);
  }
  if (a.E <= 64) return launch_topk_v<DT, 64, 1>(logits, bias, ids, weights, T, a, stream);
  if (a.E <= 256) return launch_topk_v<DT, 64, 4>(logits, bias, ids, weights, T, a, stream);
  if (a.E <= 512) return launch_topk_v<DT, 64, 8>(logits, bias, ids, weights, T, a, stream);
  return launch_topk_v<DT, 64, 16>(logits, bias, ids, weights, T, a, stream);
}
template <int DT, int L, int V>
hipError_t launch_topk_grad_v(const void *logits, const int *ids, const float *dweights, void *dlogits, int64_t T,
                              const TopkArgs &a, hipStream_t stream) {
  typedef typename Element<DT>::type E_t;
  const int64_t tokens = kWaves * (64 / L);
  hipLaunchKernelGGL((topk_grad_kernel<DT, L, V>), dim3(static_cast<unsigned>((T + tokens - 1) / tokens)), dim3(kWaves * 64), 0,
                     stream, static_cast<const E_t *>(logits), ids, dweights, static_cast<E_t *>(dlogits), T, a);
  return hipGetLastError();
}
template <int DT>
hipError_t launch_topk_grad_dt(const void *logits, const int *ids, const float *dweights, void *dlogits, int64_t T,
                               const TopkArgs &a, hipStream_t stream) {
  if (a.k <= 16) {
    if (a.E <= 32) return launch_topk_grad_v<DT, 16, 2>(logits, ids, dweights, dlogits, T, a, stream);
    if (a.E <= 64) return launch_topk_grad_v<DT, 16, 4>(logits, ids, dweights, dlogits, T, a, stream);
    if (a.E <= 128) return launch_topk_grad_v<DT, 16, 8>(logits, ids, dweights, dlogits, T, a, stream);
    if (a.E <= 256) return launch_topk_grad_v<DT, 16, 16>(logits, ids, dweights, dlogits, T, a, stream);
  }
  if (a.E <= 64) return launch_topk_grad_v<DT, 64, 1>(logits, ids, dweights, dlogits, T, a, stream);
  if (a.E <= 256) return launch_topk_grad_v<DT, 64, 4>(logits, ids, dweights, dlogits, T, a, stream);
  if (a.E <= 512) return launch_topk_grad_v<DT, 64, 8>(logits, ids, dweights, dlogits, T, a, stream);
  return launch_topk_grad_v<DT, 64, 16>(logits, ids, dweights, dlogits, T, a, stream);
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

// One workgroup (and launch) for as many slots as it sorts sooner than two launches do
// (E = 256, us with one / two: 1024 slots 4.6 / 6.7, 4096 8.9 / 7.7), then 512 slots to a
// workgroup, up to 128 of them, as each reads all the others' counts (131072 slots: 10.4
// us with 64, 9.7 with 128, 11.2 with 256).
int route_sort_blocks(int64_t slots) {
  if (slots <= 2048) return 1;
  const int64_t b = (slots + 511) / 512;
  return static_cast<int>(b < 128 ? b : 128);
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
