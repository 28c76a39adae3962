// Router top-k and the grouping of rows by the matrix they take.
//
// Top-k: a token's E logits lie in V registers of L lanes (element v L +
// lane). Each of the k rounds takes the largest (logit, lowest index) by a
// maximum over the lane's V keys and log2 L exchanges between lanes,
// and clears the taken one. A key is the logit mapped to an integer of the
// same order with the inverted index behind it, so one integer maximum
// decides ties: 32 bits for the 16-bit types, 64 for fp32.
//
// Grouping is a stable counting sort. A block of up to kSlots slots ranks
// its slots within their group by ballots over the bits of the group number
// (lanes with equal ids find each other), adds the counts of the waves
// before, and the counts of all blocks before. Up to kSlots slots are one
// launch; more are two: the blocks' counts, then the placement, in which
// every block adds up the counts itself (a grid-wide prefix without a third
// launch or a wait between blocks). Nothing depends on the order in which
// blocks run, so neither does the result.
//
// Measured: 16384 tokens, 8 of 128: 18 us, 131072 61, 524288 249; rows
// grouped by 64 ids: 2^14 12 us, 2^20 19, 2^22 83, 2^24 826. The sums over
// all blocks' counts grow with the square of the blocks, times the groups:
// 2^24 rows by 1024 ids take 12 ms.
#include <math.h>

#include "op16.h"
#include "row_groups.h"

namespace qw {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kSlots = 2048;  // slots of one block

// ---- top-k keys ----------------------------------------------------------

// Integer with the order of the float's value; NaN and -inf give 0.
__device__ inline uint32_t ordered32(float f) {
  if (!(f > -INFINITY)) return 0u;
  const uint32_t u = __builtin_bit_cast(uint32_t, f + 0.0f);  // -0 counts as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ inline float from_ordered32(uint32_t k) {
  return __builtin_bit_cast(float, (k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// The largest of v over the L lanes of a token, in every one of them. Row
// operations and half swaps in place of lane permutes through LDS, whose
// latency would be most of the time of a round.
template <int CTRL, typename T>
__device__ inline T row_max(T v) {
  T o;
  if constexpr (sizeof(T) == 8) {
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, 0xF, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, 0xF, 0xF, true);
    o = (T)hi << 32 | lo;
  } else {
    o = (T)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
  }
  return o > v ? o : v;
}
template <bool HALVES, typename T>
__device__ inline T swap_max(T v) {
  auto swap = [](uint32_t w, uint32_t &a, uint32_t &b) {
    if constexpr (HALVES) {
      const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
      a = r[0], b = r[1];
    } else {
      const auto r = __builtin_amdgcn_permlane16_swap(w, w, false, false);
      a = r[0], b = r[1];
    }
  };
  uint32_t a, b;
  swap((uint32_t)v, a, b);
  if constexpr (sizeof(T) == 8) {
    uint32_t c, d;
    swap((uint32_t)(v >> 32), c, d);
    const T x = (T)c << 32 | a, y = (T)d << 32 | b;
    return x > y ? x : y;
  } else {
    return a > b ? a : b;
  }
}
template <int L, typename T>
__device__ inline T lanes_max(T v) {
  v = row_max<0xB1>(v);              // quad permute 1 0 3 2
  v = row_max<0x4E>(v);              // quad permute 2 3 0 1
  v = row_max<0x141>(v);             // mirror in half rows
  if constexpr (L >= 16) v = row_max<0x140>(v);  // mirror in rows
  if constexpr (L >= 32) v = swap_max<false>(v);
  if constexpr (L >= 64) v = swap_max<true>(v);
  return v;
}

// 16-bit logits: the upper half of the fp32 pattern (bf16), or the fp16
// pattern itself, above the inverted index.
template <int DT>
struct Keys {
  using key_t = uint32_t;
  static __device__ key_t make(const void *p, size_t i, int e) {
    const uint32_t h = reinterpret_cast<const uint16_t *>(p)[i];
    const uint32_t mag = h & 0x7FFFu, inf = DT == QW_DT_BF16 ? 0x7F80u : 0x7C00u;
    if (mag > inf || h == (inf | 0x8000u)) return 0u;  // NaN, -inf
    const uint32_t o = (mag && (h & 0x8000u)) ? 0x8000u - mag : 0x8000u + mag;  // >= 1
    return (o << 16) | (0xFFFFu - (uint32_t)e);
  }
  static __device__ int index(key_t k) { return (int)(0xFFFFu - (k & 0xFFFFu)); }
  static __device__ float value(key_t k) {
    const uint32_t o = k >> 16;
    const uint32_t h = o < 0x8000u ? (0x8000u - o) | 0x8000u : o - 0x8000u;
    return DT == QW_DT_BF16 ? __builtin_bit_cast(float, h << 16) : f16_bits_to_f32((uint16_t)h);
  }
};
template <>
struct Keys<QW_DT_F32> {
  using key_t = unsigned long long;
  static __device__ key_t make(const void *p, size_t i, int e) {
    const uint32_t o = ordered32(reinterpret_cast<const float *>(p)[i]);
    return o ? ((key_t)o << 32) | (0xFFFFFFFFu - (uint32_t)e) : 0ull;
  }
  static __device__ int index(key_t k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }
  static __device__ float value(key_t k) { return from_ordered32((uint32_t)(k >> 32)); }
};

struct RouteArgs {
  const void *logits;
  int32_t *ids;
  float *weights;
  int T, E, k, normalize;
};

// The top-k of tokens t0 .. t0 + count - 1 by one block; ids also to the
// LDS array sid where the block places them itself.
template <int DT, int L, int V>
__device__ inline void topk_tokens(const RouteArgs &a, int t0, int count, int32_t *sid) {
  using KT = Keys<DT>;
  const int sub = threadIdx.x % L;
  for (int i = threadIdx.x / L; i < count; i += kThreads / L) {
    const int t = t0 + i;
    typename KT::key_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + sub;
      key[v] = e < a.E ? KT::make(a.logits, (size_t)t * a.E + e, e) : 0;
    }
    // weight denominators over all experts need every exponential
    float top = 0.0f, sum = 0.0f;
    int id = -1;          // this lane's choice (lane j of the token keeps choice j)
    float w = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      typename KT::key_t best = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) best = key[v] > best ? key[v] : best;
      best = lanes_max<L>(best);
      const float val = KT::value(best);
      if (j == 0) {
        top = val;
        if (!a.normalize) {
#pragma unroll
          for (int v = 0; v < V; ++v) sum += key[v] ? expf(KT::value(key[v]) - top) : 0.0f;
#pragma unroll
          for (int d = L / 2; d; d >>= 1) sum += __shfl_xor(sum, d, L);
        }
      }
      const float e = best ? expf(val - top) : 0.0f;
      if (a.normalize) sum += e;
      if (sub == j) {
        id = best ? KT::index(best) : -1;
        w = e;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = key[v] == best ? 0 : key[v];
    }
    if (sub < a.k) {
      const size_t o = (size_t)t * a.k + sub;
      a.ids[o] = id;
      a.weights[o] = id >= 0 ? w / sum : 0.0f;
      if (sid) sid[i * a.k + sub] = id;
    }
  }
}

// ---- scores, bias and groups ---------------------------------------------
//
// The choice of qw_route_scored. A token's lanes are dealt to its groups of
// experts: with the number of groups rounded up to a power of two, lane `sub`
// belongs to group sub / P and holds the experts sub % P, sub % P + P, ... of
// it, so a group's largest and second come from log2 P exchanges, and with
// one group the layout is that of the top-k above.
//
// The order has to be that of 64-bit numbers: sigmoids of logits that differ in
// fp32 agree in fp32 as soon as they come near 1, and a bias of 0.1 leaves
// scores of 1e-4 three digits. So the choice is made in fp32 first, and where
// two values that it depends on are nearer to each other than fp32 can tell
// (unsure), it is made again in 64 bits: some tokens in a hundred with fp32
// logits, all with equal choices. Without a bias a score's order is its logit's,
// and only sums of two are unsure, and logits whose scores may be one 64-bit number
// (may_level). A token's choice is that of its own 64-bit scores, whichever path
// its wave takes. 16384 tokens, 8 of 256 in 4 of 8 groups:
// 39 us, all of it in 64 bits 52.
//
// The chosen experts' scores are computed again from their logits, one a lane
// and in 64 bits, rather than kept.

struct ScoredArgs {
  const void *logits;
  const float *bias;
  int32_t *ids;
  float *weights;
  float scale;
  int T, E, k, normalize;
  int score, by;
  int groups, top_groups, group_size;
};

// Integer with the order of the number; NaN and -inf give 0.
__device__ inline unsigned long long ordered64(double f) {
  if (!(f > -INFINITY)) return 0ull;
  const unsigned long long u = __builtin_bit_cast(unsigned long long, f + 0.0);  // -0 counts as 0
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ inline double from_ordered64(unsigned long long k) {
  return __builtin_bit_cast(double, (k >> 63) ? (k & ~(1ull << 63)) : ~k);
}

// Order of a 16-bit logit (not NaN or -inf) as an integer of 16 bits, >= 1.
template <int DT>
__device__ inline uint32_t ordered16(float x) {
  const uint32_t h = DT == QW_DT_BF16 ? __builtin_bit_cast(uint32_t, x) >> 16 : (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x);
  const uint32_t mag = h & 0x7FFFu;
  return mag && (h & 0x8000u) ? 0x8000u - mag : 0x8000u + mag;
}

template <int DT>
__device__ inline float logit_at(const void *p, size_t i) {
  if constexpr (DT == QW_DT_F32) return reinterpret_cast<const float *>(p)[i];
  const uint32_t h = reinterpret_cast<const uint16_t *>(p)[i];
  return DT == QW_DT_BF16 ? __builtin_bit_cast(float, h << 16) : f16_bits_to_f32((uint16_t)h);
}

// What the lanes of a token know of it. Lane `sub` holds the experts
// first + v P of its group.
template <int L, int V>
struct TokenLanes {
  int sub, P, group, first;
  __device__ TokenLanes(const ScoredArgs &a) {
    sub = threadIdx.x % L;
    P = L;  // lanes of a group
    while (L / P < a.groups) P /= 2;
    group = sub / P;
    first = group * a.group_size + sub % P;
  }
  __device__ bool has(const ScoredArgs &a, int v) const { return group < a.groups && v * P + sub % P < a.group_size; }
};

__device__ inline double score64(const ScoredArgs &a, float l, float most, double sum) {
  return a.score == QW_ROUTE_SOFTMAX ? exp((double)l - (double)most) / sum : 1.0 / (1.0 + exp(-(double)l));
}
template <int L>
__device__ inline double sum_of(double v) {
#pragma unroll
  for (int d = L / 2; d; d >>= 1) v += __shfl_xor(v, d, L);
  return v;
}
// The sum of the exponentials of all of a token's logits.
template <int L, int V>
__device__ inline double sum64(const float (&x)[V], float most) {
  double sum = 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v) sum += x[v] > -INFINITY ? exp((double)x[v] - (double)most) : 0.0;
  return sum_of<L>(sum);
}

// The choice in 64 bits: this lane's expert (lane j of the token keeps choice
// j), -1 where there is none.
template <int L, int V>
__device__ inline int choose64(const ScoredArgs &a, const TokenLanes<L, V> &t, const float (&x)[V], const float (&bias)[V], float most) {
  typedef unsigned long long key_t;
  const double sum = a.score == QW_ROUTE_SOFTMAX ? sum64<L>(x, most) : 1.0;
  key_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    key[v] = 0;
    if (x[v] > -INFINITY) key[v] = ordered64(score64(a, x[v], most, sum) + (double)bias[v]);
  }
  if (a.top_groups < a.groups) {
    key_t one = 0, two = 0;  // the group's largest and second
#pragma unroll
    for (int v = 0; v < V; ++v) {
      two = max(two, min(one, key[v]));
      one = max(one, key[v]);
    }
    for (int d = t.P / 2; d; d >>= 1) {
      const key_t f = __shfl_xor(one, d, L), s = __shfl_xor(two, d, L);
      two = max(min(one, f), max(two, s));
      one = max(one, f);
    }
    key_t value = one;
    if (a.by == QW_GROUP_TOP2 && two) value = ordered64(from_ordered64(one) + from_ordered64(two));
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
      const key_t o = __shfl(value, g * t.P, L);
      before += o > value || (o == value && g < t.group);
    }
    if (before >= a.top_groups) {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = 0;
    }
  }
  int id = -1;
  for (int j = 0; j < a.k; ++j) {
    key_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = key[v] > best ? key[v] : best;
    best = lanes_max<L>(best);
    uint32_t at = 0;  // the inverted number of the lowest expert that has it
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (best && key[v] == best) at = max(at, ~(uint32_t)(t.first + v * t.P));
    at = lanes_max<L>(at);
    if (t.sub == j && best) id = (int)~at;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (~(uint32_t)(t.first + v * t.P) == at) key[v] = 0;
  }
  return id;
}

// How near two fp32 choices may lie and still be unsure: more than both are off by
// together (two groups' sums: than half of it, so each group brings one).
// A sigmoid is off by |l| s (1 - s) 2^-23 + s (1 - s) 2^-23 (the exponential's
// argument, rounded twice, and its step) and two roundings of numbers up to 1: less
// than 3e-7. Softmax scores share the error of their sum, V - 1 + log2 L half steps.
// Their exponentials, 2.5 d + 2 half steps each at a distance of d from the largest,
// weigh in by their scores, which are 1 together at most: 11 half steps for two
// scores and their sum, 14 for four; the quotient and the product round once each.
// A choice is rounded once more behind the bias, a sum of two twice: `size` is what
// the terms add up to without their signs (terms that cancel keep their errors).
template <int L, int V>
__device__ inline float unsure(const ScoredArgs &a, float size) {
  constexpr int kLog = L == 16 ? 4 : L == 32 ? 5 : 6;
  return (a.score == QW_ROUTE_SIGMOID ? 8e-7f : (float)(V - 1 + kLog + 16) * 0x1p-24f) + 0x1p-22f * size;
}

// Without a bias the logits have the order of the scores, but the scores' 64-bit
// numbers may be equal where the logits are not, and then the lower expert comes
// first: sigmoids above 37 are all 1, what lies below -745 (softmax: that far below
// the largest) is 0, and logits next to 0 have one score. Whether a logit may be one
// of those, with room. A pair of others has two numbers: sigmoids of fp32 logits up
// to 20 are 4e-15 apart, logits of 2^-12 and more 2^-36.
__device__ inline bool may_level(const ScoredArgs &a, float l, float most) {
  return (a.score == QW_ROUTE_SIGMOID ? l > 20.0f || l < -700.0f : l - most < -700.0f) || fabsf(l) < 0x1p-12f;
}

// The same with 32-bit keys; chosen[j] (LDS) receives choice j. Returns whether
// it is the choice in 64 bits for sure.
//
// A round is a maximum over the lane's keys and the lanes, and the lane that has
// it stores its number and clears it. Keys of 16-bit logits hold the inverted
// number behind the logit, so no two are equal; equal keys of the other kinds
// show in the count of what k rounds have cleared.
template <int DT, int L, int V>
__device__ inline bool choose32(const ScoredArgs &a, const TokenLanes<L, V> &t, const float (&x)[V], const float (&bias)[V], float most, int32_t *chosen) {
  const bool sums = a.top_groups < a.groups && a.by == QW_GROUP_TOP2;
  const bool scores = a.bias || sums;  // else the logits have the order
  bool sure = true;
  float c[V];
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = x[v];
  if (scores) {
    float inv = 1.0f;
    if (a.score == QW_ROUTE_SOFTMAX) {
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        c[v] = x[v] > -INFINITY ? __expf(x[v] - most) : 0.0f;
        sum += c[v];
      }
#pragma unroll
      for (int d = L / 2; d; d >>= 1) sum += __shfl_xor(sum, d, L);
      inv = 1.0f / sum;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float s = a.score == QW_ROUTE_SOFTMAX ? c[v] * inv : __frcp_rn(1.0f + __expf(-x[v]));
      const float choice = s + bias[v];
      c[v] = x[v] > -INFINITY && choice > -INFINITY ? choice : -INFINITY;  // NaN is taken as -inf
    }
  }
  if (a.top_groups < a.groups) {
    float one = -INFINITY, two = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      two = fmaxf(two, fminf(one, c[v]));
      one = fmaxf(one, c[v]);
    }
    for (int d = t.P / 2; d; d >>= 1) {
      const float f = __shfl_xor(one, d, L), s = __shfl_xor(two, d, L);
      two = fmaxf(fminf(one, f), fmaxf(two, s));
      one = fmaxf(one, f);
    }
    const float value = sums && two > -INFINITY ? one + two : one;
    const float mine = unsure<L, V>(a, fabsf(one) + (sums && two > -INFINITY ? fabsf(two) : 0.0f));
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
      const float o = __shfl(value, g * t.P, L);
      const float near = !scores ? -1.0f : mine + (a.bias ? __shfl(mine, g * t.P, L) : mine);
      before += o > value || (o == value && g < t.group);
      // (a group that has no expert left is behind all others in any case)
      if (g != t.group && value > -INFINITY && o > -INFINITY && !(fabsf(o - value) > near)) sure = false;
    }
    const bool level = !scores && value > -INFINITY && may_level(a, value, most);
    if (__any(level)) {
      for (int g = 0; g < a.groups; ++g)
        if (__shfl((int)level, g * t.P, L) && level && g != t.group) sure = false;
    }
    if (before >= a.top_groups) {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = -INFINITY;
    }
  }
  // without a bias the order within the groups is the logits'
  const bool unique = DT != QW_DT_F32 && !a.bias;
  uint32_t key[V];
  int left = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t o = ordered32(a.bias ? c[v] : c[v] > -INFINITY ? x[v] : -INFINITY);
    key[v] = o;
    if constexpr (DT != QW_DT_F32)
      if (unique && o) key[v] = (ordered16<DT>(x[v]) << 16) | (0xFFFFu - (uint32_t)(t.first + v * t.P));
    left += key[v] != 0;
  }
  if (t.sub < a.k) chosen[t.sub] = -1;
  float last = INFINITY;
  int taken = 0;
  const int rounds = a.bias ? a.k + 1 : a.k;  // the first that is not chosen, too
  for (int j = 0; j < rounds; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    best = lanes_max<L>(best);
    if (a.bias && best) {
      const float value = from_ordered32(best);
      if (!(last - value > unsure<L, V>(a, fabsf(value)))) sure = false;  // j = 0: infinity, and NaN where the value is infinite too
      last = value;
    }
    if (j == a.k || __all(best == 0)) break;
    int at = -1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool is = key[v] == best;
      at = is ? v : at;
      key[v] = is ? 0 : key[v];
    }
    if (best) {
      ++taken;
      if (at >= 0) chosen[j] = t.first + at * t.P;
    }
  }
  if (!unique) {
    int now = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) now += key[v] != 0;
    int gone = left - now;
#pragma unroll
    for (int d = L / 2; d; d >>= 1) gone += __shfl_xor(gone, d, L);
    if (gone != taken) sure = false;
  }
  return sure;
}

template <int DT, int L, int V, int NT>
__device__ inline void choose_tokens(const ScoredArgs &a, int t0, int count, int32_t *sid) {
  const TokenLanes<L, V> lanes(a);
  const int sub = lanes.sub;
  constexpr int kSide = NT / L;  // tokens side by side
  float next[V];
  auto load = [&](int i) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      next[v] = i < count && lanes.has(a, v) ? logit_at<DT>(a.logits, (size_t)(t0 + i) * a.E + lanes.first + v * lanes.P) : -INFINITY;
  };
  load(threadIdx.x / L);
  float bias[V];
#pragma unroll
  for (int v = 0; v < V; ++v) bias[v] = a.bias && lanes.has(a, v) ? a.bias[lanes.first + v * lanes.P] : 0.0f;
  for (int i = threadIdx.x / L; i < count; i += kSide) {
    const int t = t0 + i;
    float x[V];
    float most = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = next[v] > -INFINITY ? next[v] : -INFINITY;  // NaN is taken as -inf
      most = fmaxf(most, x[v]);
    }
    load(i + kSide);
    const bool softmax = a.score == QW_ROUTE_SOFTMAX;
    if (softmax) {
#pragma unroll
      for (int d = L / 2; d; d >>= 1) most = fmaxf(most, __shfl_xor(most, d, L));
    }
    int32_t *const chosen = sid + i * a.k;
    bool sure = choose32<DT, L>(a, lanes, x, bias, most, chosen) && !(softmax && most == INFINITY);  // such a row has no scores
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    int id = sub < a.k ? chosen[sub] : -1;
    if (!a.bias) {  // a choice and the next, or the last and the first that is none, may have one score
      const int lane = threadIdx.x & 63;
      const bool level = id >= 0 && may_level(a, logit_at<DT>(a.logits, (size_t)t * a.E + id), most);
      const unsigned long long others = __ballot(id >= 0 && !level);
      if (level && (sub == a.k - 1 || !((others >> ((lane + 1) & 63)) & 1))) sure = false;
    }
    const unsigned long long doubts = __ballot(!sure);
    if (doubts) {  // of one of the wave's tokens: the others keep their choice
      const int id64 = choose64<L>(a, lanes, x, bias, most);
      constexpr unsigned long long kToken = L == 64 ? ~0ull : (1ull << (L % 64)) - 1;
      if ((doubts >> ((threadIdx.x & 63) / L * L)) & kToken) {
        id = id64;
        if (sub < a.k) chosen[sub] = id;
      }
    }
    // normalised weights do not need the sum over all experts
    const double sum = softmax && !a.normalize ? sum64<L>(x, most) : 1.0;
    const double w = id >= 0 ? score64(a, logit_at<DT>(a.logits, (size_t)t * a.E + id), most, sum) : 0.0;
    double factor = (double)a.scale;
    if (a.normalize) {
      const double total = sum_of<L>(w);
      factor = total > 0.0 ? factor / total : 0.0;
    }
    if (sub < a.k) {
      const size_t o = (size_t)t * a.k + sub;
      a.ids[o] = id;
      a.weights[o] = id >= 0 ? (float)(w * factor) : 0.0f;
    }
  }
}

// ---- grouping ------------------------------------------------------------

// LDS of one block: the slots' ids, the running base of every group (one
// more for the rows of none), and the counts of each wave.
struct GroupLds {
  int32_t *sid;   // [kSlots]
  int32_t *base;  // [G + 1]
  int32_t *wave;  // [kWaves][G + 1]
};

__device__ inline GroupLds group_lds(int32_t *smem, int G) {
  return GroupLds{smem, smem + kSlots, smem + kSlots + (G + 1)};
}
constexpr size_t group_lds_bytes(int G) {
  return (size_t)(kSlots + (kWaves + 1) * (G + 1)) * sizeof(int32_t);
}

// Counts of the block's slots per group (G: none) into base.
template <int NT = kThreads>
__device__ inline void count_slots(const GroupLds &l, int slots, int G) {
  for (int g = threadIdx.x; g <= G; g += NT) l.base[g] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < slots; i += NT) {
    const int id = l.sid[i];
    atomicAdd(&l.base[(uint32_t)id < (uint32_t)G ? id : G], 1);
  }
  __syncthreads();
}

// In place: counts per bin to the exclusive prefix sum over the G + 1 bins.
// tmp: kWaves words.
__device__ inline void exclusive_scan(int32_t *v, int bins, int32_t *tmp) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int carry = 0;
  for (int g0 = 0; g0 < bins; g0 += kThreads) {
    const int g = g0 + threadIdx.x;
    const int own = g < bins ? v[g] : 0;
    int upto = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(upto, d, 64);
      if (lane >= d) upto += o;
    }
    if (lane == 63) tmp[wv] = upto;
    __syncthreads();
    int pre = carry, all = carry;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wv) pre += tmp[w];
      all += tmp[w];
    }
    if (g < bins) v[g] = pre + upto - own;
    carry = all;
    __syncthreads();
  }
}

// Places the block's slots (ids in sid, first slot s0): base holds the
// position of the block's first row of each group, on return of its next.
__device__ inline void place_slots(const GroupLds &l, int slots, int s0, int G, int32_t *rows) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int bits = 0;
  while ((1 << bits) <= G) ++bits;  // bits of the bin numbers 0..G
  for (int i0 = 0; i0 < slots; i0 += kThreads) {
    for (int g = threadIdx.x; g < kWaves * (G + 1); g += kThreads) l.wave[g] = 0;
    __syncthreads();
    const int i = i0 + threadIdx.x;
    const bool live = i < slots;
    int bin = G;
    if (live) {
      const int id = l.sid[i];
      bin = (uint32_t)id < (uint32_t)G ? id : G;
    }
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((bin >> b) & 1);
      same &= ((bin >> b) & 1) ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (live && rank == 0) l.wave[wv * (G + 1) + bin] = __popcll(same);
    __syncthreads();
    for (int g = threadIdx.x; g <= G; g += kThreads) {
      int at = l.base[g];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const int c = l.wave[w * (G + 1) + g];
        l.wave[w * (G + 1) + g] = at;
        at += c;
      }
      l.base[g] = at;
    }
    __syncthreads();
    if (live) rows[l.wave[wv * (G + 1) + bin] + rank] = s0 + i;
    __syncthreads();
  }
}

struct GroupArgs {
  const int32_t *ids;  // read where no router wrote them
  int32_t *offsets, *rows;
  int32_t *counts;     // [blocks][G] of a two-launch call
  int n, G;
  int per;             // slots of a block
  int blocks;
};

// The whole grouping of one block's slots (n <= kSlots).
__device__ inline void group_alone(const GroupArgs &g, const GroupLds &l) {
  count_slots(l, g.n, g.G);
  exclusive_scan(l.base, g.G + 1, l.wave);
  for (int i = threadIdx.x; i <= g.G; i += kThreads) g.offsets[i] = l.base[i];
  __syncthreads();
  place_slots(l, g.n, 0, g.G, g.rows);
}

template <int NT = kThreads>
__device__ inline void write_counts(const GroupArgs &g, const GroupLds &l, int slots) {
  count_slots<NT>(l, slots, g.G);
  for (int i = threadIdx.x; i < g.G; i += NT) g.counts[(size_t)blockIdx.x * g.G + i] = l.base[i];
}

template <int DT, int L, int V>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a, GroupArgs g) {
  extern __shared__ int32_t smem[];
  const GroupLds l = group_lds(smem, g.G);
  const int tokens = g.per / a.k;  // per is a multiple of k
  const int t0 = blockIdx.x * tokens;
  const int count = min(tokens, a.T - t0);
  topk_tokens<DT, L, V>(a, t0, count, l.sid);
  __syncthreads();
  if (g.blocks == 1)
    group_alone(g, l);
  else
    write_counts(g, l, count * a.k);
}

// NT: threads of a block; more than kThreads only where several blocks run.
template <int DT, int L, int V, int NT>
__global__ __launch_bounds__(NT) void scored_kernel(ScoredArgs a, GroupArgs g) {
  extern __shared__ int32_t smem[];
  const GroupLds l = group_lds(smem, g.G);
  const int tokens = g.per / a.k;  // per is a multiple of k
  const int t0 = blockIdx.x * tokens;
  const int count = min(tokens, a.T - t0);
  choose_tokens<DT, L, V, NT>(a, t0, count, l.sid);
  __syncthreads();
  if (NT == kThreads && g.blocks == 1)
    group_alone(g, l);
  else
    write_counts<NT>(g, l, count * a.k);
}

// First launch of qw_group_rows: everything for one block, else its counts.
__global__ __launch_bounds__(kThreads) void group_kernel(GroupArgs g) {
  extern __shared__ int32_t smem[];
  const GroupLds l = group_lds(smem, g.G);
  const int s0 = blockIdx.x * g.per, slots = min(g.per, g.n - s0);
  for (int i = threadIdx.x; i < slots; i += kThreads) l.sid[i] = g.ids[s0 + i];
  __syncthreads();
  if (g.blocks == 1)
    group_alone(g, l);
  else
    write_counts(g, l, slots);
}

// Second launch: the block's bases from the counts of all blocks, then the
// placement. The threads are dealt over (part of the blocks, group), so the
// reads of one part are consecutive and the parts run side by side.
__global__ __launch_bounds__(kThreads) void place_kernel(GroupArgs g) {
  extern __shared__ int32_t smem[];
  const GroupLds l = group_lds(smem, g.G);
  const int G = g.G, b = blockIdx.x;
  const int s0 = b * g.per, slots = min(g.per, g.n - s0);
  for (int i = threadIdx.x; i < slots; i += kThreads) l.sid[i] = g.ids[s0 + i];
  int32_t *const total = l.wave, *const mine = l.wave + (G + 1);  // all blocks; blocks before b
  for (int i = threadIdx.x; i <= G; i += kThreads) total[i] = mine[i] = 0;
  __syncthreads();
  const int parts = max(1, kThreads / G);
  const int part = threadIdx.x / G;
  if (G <= kThreads ? part < parts : true) {
    for (int e = G <= kThreads ? threadIdx.x % G : threadIdx.x; e < G; e += kThreads) {
      int all = 0, before = 0;
#pragma unroll 16
      for (int q = G <= kThreads ? part : 0; q < g.blocks; q += parts) {
        const int c = g.counts[(size_t)q * G + e];
        all += c;
        before += q < b ? c : 0;
      }
      atomicAdd(&total[e], all);  // integer sums: the order does not matter
      atomicAdd(&mine[e], before);
    }
  }
  __syncthreads();
  // bin G (rows of no group): behind all groups; before this block lie s0
  // slots, less those that are in a group
  for (int i = threadIdx.x; i <= G; i += kThreads) l.base[i] = i < G ? total[i] : 0;
  __syncthreads();
  exclusive_scan(l.base, G + 1, l.wave + 2 * (G + 1));
  if (b == 0)
    for (int i = threadIdx.x; i <= G; i += kThreads) g.offsets[i] = l.base[i];
  __syncthreads();
  if (threadIdx.x == 0) l.wave[2 * (G + 1) + kWaves] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < G; i += kThreads) atomicAdd(&l.wave[2 * (G + 1) + kWaves], mine[i]);
  __syncthreads();
  const int grouped_before = l.wave[2 * (G + 1) + kWaves];
  for (int i = threadIdx.x; i <= G; i += kThreads) l.base[i] += i < G ? mine[i] : s0 - grouped_before;
  __syncthreads();
  place_slots(l, slots, s0, G, g.rows);
}

// Rows of a block of qw_group_rows: all of them up to kSlots, else 512 until
// the counts that every block adds up would be the larger cost, at most
// kSlots.
int block_rows(long long n) {
  long long per = n <= kSlots ? n : 512;
  while (per < kSlots && n > per * 256) per *= 2;
  return (int)per;
}

// Lanes a token takes in the top-k: enough that a lane holds at most 8
// logits (16 beyond 512 experts) and that every choice has a lane to keep
// it; fewer lanes mean more tokens side by side and fewer exchanges.
int topk_lanes(int E, int k) {
  if (E <= 32 && k <= 8) return 8;
  if (E <= 128 && k <= 16) return 16;
  return E <= 256 ? 32 : 64;
}

// Slots of a block of the router: all of them where they are at most kSlots
// and the top-k takes few passes; else two passes of the top-k a block (16384
// tokens of 8 in 128: 10 us, 17 with twice as many), more where there would
// be over 256 blocks, at most kSlots. A multiple of k.
int block_slots(int T, int E, int k) {
  const int pass = kThreads / topk_lanes(E, k);
  if (T <= 4 * pass && (long long)T * k <= kSlots) return T * k;
  long long tokens = 2 * pass;
  while (2 * tokens * k <= kSlots && T > tokens * 256) tokens *= 2;
  while (tokens > 1 && tokens * k > kSlots) tokens /= 2;
  return (int)(tokens * k);
}


// Lanes a token takes in the choice by scores, and the experts that a lane
// holds: as in the top-k, with a lane at least for every group.
int scored_lanes(int E, int k, int groups) {
  int lanes = topk_lanes(E, k);
  lanes = lanes < 16 ? 16 : lanes;
  while (lanes < groups) lanes *= 2;
  return lanes;
}
// Slots of a block: one pass of the choice a block (64 tokens, 8 of 256: two
// launches with 4 blocks 15.7 us, one with a block of 4 passes 34), more
// where there would be over 256 blocks, at most kSlots.
int scored_slots(int T, int E, int k, int groups) {
  const int pass = kThreads / scored_lanes(E, k, groups);
  if (T <= pass) return T * k;
  long long tokens = pass;
  while (2 * tokens * k <= kSlots && T > tokens * 256) tokens *= 2;
  while (tokens > 1 && tokens * k > kSlots) tokens /= 2;
  return (int)(tokens * k);
}
int scored_held(int E, int groups, int lanes) {
  int per = lanes;  // lanes of a group
  while (lanes / per < groups) per /= 2;
  const int held = (E / groups + per - 1) / per;
  return held <= 4 ? 4 : held <= 8 ? 8 : held <= 16 ? 16 : 32;
}

size_t counts_bytes(long long n, int per, int G) {
  return n <= per ? 0 : (size_t)((n + per - 1) / per) * (size_t)G * sizeof(int32_t);
}

qw_status launch_place(const GroupArgs &g, hipStream_t s) {
  if (g.blocks == 1) return QW_OK;
  QW_HIP_TRY(launch(place_kernel, g.blocks, kThreads, group_lds_bytes(g.G), s, g));
  return QW_OK;
}

template <int DT>
qw_status launch_route(const RouteArgs &a, const GroupArgs &g, hipStream_t s) {
  const size_t lds = group_lds_bytes(g.G);
  const int lanes = topk_lanes(a.E, a.k);
#define QW_ROUTE(L, V)                                                                \
  if (lanes == (L) && a.E <= (L) * (V)) {                                             \
    QW_HIP_TRY(launch(route_kernel<DT, L, V>, g.blocks, kThreads, lds, s, a, g));     \
    return launch_place(g, s);                                                        \
  }
  QW_ROUTE(8, 4)
  QW_ROUTE(16, 4)
  QW_ROUTE(16, 8)
  QW_ROUTE(32, 8)
  QW_ROUTE(64, 8)
  QW_ROUTE(64, 16)
#undef QW_ROUTE
  return QW_ERR_UNSUPPORTED;
}

template <int DT>
qw_status launch_scored(const ScoredArgs &a, const GroupArgs &g, hipStream_t s) {
  const size_t lds = group_lds_bytes(g.G);
  const int lanes = scored_lanes(a.E, a.k, a.groups), held = scored_held(a.E, a.groups, lanes);
  // blocks of several passes have twice the threads where their registers allow
  // it: a pass is a chain of exchanges, which other waves fill (16384 tokens, 8
  // of 256: 39 us, with 512 threads 46)
  const bool twice = g.blocks > 1 && g.per / a.k > kThreads / lanes;
#define QW_SCORED(L, V)                                                                          \
  if (lanes == (L) && held == (V)) {                                                             \
    if constexpr (V <= 8) {                                                                      \
      if (twice) {                                                                               \
        QW_HIP_TRY(launch(scored_kernel<DT, L, V, 2 * kThreads>, g.blocks, 2 * kThreads, lds, s, a, g)); \
        return launch_place(g, s);                                                               \
      }                                                                                          \
    }                                                                                            \
    QW_HIP_TRY(launch(scored_kernel<DT, L, V, kThreads>, g.blocks, kThreads, lds, s, a, g));     \
    return launch_place(g, s);                                                                   \
  }
  QW_SCORED(16, 4)
  QW_SCORED(16, 8)
  QW_SCORED(16, 16)
  QW_SCORED(32, 4)
  QW_SCORED(32, 8)
  QW_SCORED(32, 16)
  QW_SCORED(64, 4)
  QW_SCORED(64, 8)
  QW_SCORED(64, 16)
  QW_SCORED(64, 32)
#undef QW_SCORED
  return QW_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace qw

extern "C" {

size_t qw_group_rows_workspace_bytes(int n, int G) {
  if (n < 1 || n > QW_MAX_ROWS || G < 1 || G > QW_MAX_GROUPS) return 0;
  return qw::counts_bytes(n, qw::block_rows(n), G);
}

size_t qw_route_workspace_bytes(int T, int E, int top_k) {
  if (T < 1 || E < 1 || E > QW_MAX_GROUPS || top_k < 1 || top_k > E || top_k > QW_MAX_TOPK) return 0;
  const long long n = (long long)T * top_k;
  return n <= QW_MAX_ROWS ? qw::counts_bytes(n, qw::block_slots(T, E, top_k), E) : 0;
}

qw_status qw_group_rows(const int32_t *ids, int n, int G, int32_t *offsets, int32_t *rows,
                        void *workspace, size_t workspace_bytes, void *stream) {
  using namespace qw;
  CallScope scope;
  if (!ids || !offsets || !rows || n < 1 || G < 1) return QW_ERR_INVALID_ARG;
  if (G > QW_MAX_GROUPS || n > QW_MAX_ROWS) return QW_ERR_UNSUPPORTED;
  const int per = block_rows(n);
  const size_t need = counts_bytes(n, per, G);
  if (need && (!workspace || workspace_bytes < need)) return QW_ERR_INVALID_ARG;
  if (!aligned16(ids) || !aligned16(offsets) || !aligned16(rows) || (need && !aligned16(workspace)))
    return QW_ERR_ALIGNMENT;
  QW_TRY(current_device(nullptr));
  GroupArgs g{};
  g.ids = ids;
  g.offsets = offsets;
  g.rows = rows;
  g.counts = reinterpret_cast<int32_t *>(workspace);
  g.n = n;
  g.G = G;
  g.per = per;
  g.blocks = (int)(((long long)n + per - 1) / per);
  QW_HIP_TRY(launch(group_kernel, g.blocks, kThreads, group_lds_bytes(G), as_stream(stream), g));
  return launch_place(g, as_stream(stream));
}

qw_status qw_route_topk(const void *logits, qw_dtype dtype, int T, int E, int top_k, int normalize,
                        int32_t *ids, float *weights, int32_t *offsets, int32_t *rows,
                        void *workspace, size_t workspace_bytes, void *stream) {
  using namespace qw;
  CallScope scope;
  if (!logits || !ids || !weights || !offsets || !rows || T < 1 || E < 1) return QW_ERR_INVALID_ARG;
  if (top_k < 1 || top_k > E || top_k > QW_MAX_TOPK) return QW_ERR_INVALID_ARG;
  if (dtype != QW_DT_F16 && dtype != QW_DT_BF16 && dtype != QW_DT_F32) return QW_ERR_INVALID_ARG;
  const long long n = (long long)T * top_k;
  if (E > QW_MAX_GROUPS || n > QW_MAX_ROWS) return QW_ERR_UNSUPPORTED;
  const int per = block_slots(T, E, top_k);
  const size_t need = counts_bytes(n, per, E);
  if (need && (!workspace || workspace_bytes < need)) return QW_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(ids) || !aligned16(weights) || !aligned16(offsets) ||
      !aligned16(rows) || (need && !aligned16(workspace)))
    return QW_ERR_ALIGNMENT;
  QW_TRY(current_device(nullptr));
  RouteArgs a{logits, ids, weights, T, E, top_k, normalize != 0};
  GroupArgs g{};
  g.ids = ids;
  g.offsets = offsets;
  g.rows = rows;
  g.counts = reinterpret_cast<int32_t *>(workspace);
  g.n = (int)n;
  g.G = E;
  g.per = per;
  g.blocks = (int)((n + per - 1) / per);
  if (dtype == QW_DT_F32) return launch_route<QW_DT_F32>(a, g, as_stream(stream));
  if (dtype == QW_DT_BF16) return launch_route<QW_DT_BF16>(a, g, as_stream(stream));
  return launch_route<QW_DT_F16>(a, g, as_stream(stream));
}

size_t qw_route_scored_workspace_bytes(int T, int E, int top_k, int n_groups) {
  if (T < 1 || E < 1 || E > QW_MAX_GROUPS || top_k < 1 || top_k > E || top_k > QW_MAX_TOPK) return 0;
  if (n_groups < 1 || n_groups > QW_MAX_EXPERT_GROUPS || E % n_groups) return 0;
  const long long n = (long long)T * top_k;
  return n <= QW_MAX_ROWS ? qw::counts_bytes(n, qw::scored_slots(T, E, top_k, n_groups), E) : 0;
}

qw_status qw_route_scored(const void *logits, qw_dtype dtype, int T, int E, int top_k, qw_route_score score,
                          const float *bias, int n_groups, int top_groups, qw_group_value group_by, int normalize,
                          float scale, int32_t *ids, float *weights, int32_t *offsets, int32_t *rows,
                          void *workspace, size_t workspace_bytes, void *stream) {
  using namespace qw;
  CallScope scope;
  if (!logits || !ids || !weights || !offsets || !rows || T < 1 || E < 1) return QW_ERR_INVALID_ARG;
  if (top_k < 1 || top_k > QW_MAX_TOPK || !is_dtype(dtype)) return QW_ERR_INVALID_ARG;
  if (score != QW_ROUTE_SOFTMAX && score != QW_ROUTE_SIGMOID) return QW_ERR_INVALID_ARG;
  if (group_by != QW_GROUP_MAX && group_by != QW_GROUP_TOP2) return QW_ERR_INVALID_ARG;
  if (n_groups < 1 || n_groups > QW_MAX_EXPERT_GROUPS || E % n_groups) return QW_ERR_INVALID_ARG;
  if (top_groups < 1 || top_groups > n_groups) return QW_ERR_INVALID_ARG;
  if (top_k > E / n_groups * top_groups || !(fabsf(scale) < INFINITY)) return QW_ERR_INVALID_ARG;
  const long long n = (long long)T * top_k;
  if (E > QW_MAX_GROUPS || n > QW_MAX_ROWS) return QW_ERR_UNSUPPORTED;
  const int per = scored_slots(T, E, top_k, n_groups);
  const size_t need = counts_bytes(n, per, E);
  if (need && (!workspace || workspace_bytes < need)) return QW_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(bias) || !aligned16(ids) || !aligned16(weights) || !aligned16(offsets) ||
      !aligned16(rows) || (need && !aligned16(workspace)))
    return QW_ERR_ALIGNMENT;
  QW_TRY(current_device(nullptr));
  ScoredArgs a{logits, bias, ids, weights, scale, T, E, top_k, normalize != 0, (int)score, (int)group_by, n_groups, top_groups, E / n_groups};
  GroupArgs g{};
  g.ids = ids;
  g.offsets = offsets;
  g.rows = rows;
  g.counts = reinterpret_cast<int32_t *>(workspace);
  g.n = (int)n;
  g.G = E;
  g.per = per;
  g.blocks = (int)((n + per - 1) / per);
  if (dtype == QW_DT_F32) return launch_scored<QW_DT_F32>(a, g, as_stream(stream));
  if (dtype == QW_DT_BF16) return launch_scored<QW_DT_BF16>(a, g, as_stream(stream));
  return launch_scored<QW_DT_F16>(a, g, as_stream(stream));
}

}  // extern "C"
