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
__device__ inline void count_slots(const GroupLds &l, int slots, int G) {
  for (int g = threadIdx.x; g <= G; g += kThreads) l.base[g] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < slots; i += kThreads) {
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

__device__ inline void write_counts(const GroupArgs &g, const GroupLds &l, int slots) {
  count_slots(l, slots, g.G);
  for (int i = threadIdx.x; i < g.G; i += kThreads) g.counts[(size_t)blockIdx.x * g.G + i] = l.base[i];
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

}  // extern "C"
