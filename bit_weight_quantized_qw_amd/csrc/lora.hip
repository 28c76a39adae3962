// Low-rank adapters of many requests beside a shared projection:
//   out[m] = base[m] + scale[a] * B_a (A_a x[m]),  a = adapter of row m
//
// Rows come grouped by adapter, so an adapter is read once for all rows of
// a tile. Two launches: t = A_a x into the workspace, then base + s B_a t.
// The first is split over K where there are few rows (a decode step would
// occupy a few CUs otherwise); each part writes its own fp32 partial sums
// and the second launch adds them in order, so the result does not depend
// on which part ran first.
//
// What bounds it: bytes. A decode step reads the used adapters, a prefill
// reads x and base and writes out; the products are small beside them. They
// come at 2.4 to 2.9 TB/s, behind chains of dependent loads.
//
// t is fp32 and the matrix cores take 16 bits, so the second product uses
// t as the sum of two 16-bit numbers, after a power of two per row that
// brings the row's largest value to 1..2 (fp16 could neither hold a large t
// nor the rest of a small one).
#include <math.h>

#include "op16.h"
#include "row_groups.h"

namespace qw {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 64;       // K elements of one step: two products
constexpr int kColTile = 256;   // output columns of a workgroup at a time

struct LoraArgs {
  const uint16_t *x, *A, *B;
  const float *scale;
  const int32_t *offsets, *rows;
  const void *base;
  void *out;
  float *part;  // [splits][n][r]
  int n, G, N, K, r;
  int splits, steps_per_split;
  int rank_tiles, col_groups, cols_per_group;
  int base_dtype, out_dtype, in_place;
};

// ---- t = A_a x -----------------------------------------------------------
// A workgroup: MR x 16 rows of one adapter, RB x 16 of its r inner values,
// one split of K. The waves take the split's 64-element steps in turn.
template <int DT, int MR, int RB>
__global__ __launch_bounds__(kThreads) void shrink_kernel(LoraArgs a) {
  using O = Op<DT>;
  __shared__ __attribute__((aligned(16))) float sum[kWaves][MR * 16][RB * 16 + 4];
  const int tid = threadIdx.x, lane = tid & 63, ln = lane & 15, lg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  int b = blockIdx.x;
  const int split = b % a.splits;
  b /= a.splits;
  const int rt0 = b % a.rank_tiles * (RB * 16);
  const RowLookup row_at(a.rows, a.n);
  const RowTile t = find_row_tile(a.offsets, a.G, a.n, MR * 16, b / a.rank_tiles);
  if (t.cnt == 0) return;
  const int K = a.K;

  // rows past the tile's end repeat its first row; inner values past r
  // repeat the last (neither is stored)
  const uint16_t *xp[MR], *ap[RB];
#pragma unroll
  for (int i = 0; i < MR; ++i) {
    const int q = i * 16 + ln;
    int m = row_at(t.p0 + (q < t.cnt ? q : 0));
    if ((uint32_t)m >= (uint32_t)a.n) m = 0;
    xp[i] = a.x + (size_t)m * K + lg * 16;
  }
#pragma unroll
  for (int j = 0; j < RB; ++j)
    ap[j] = a.A + ((size_t)t.g * a.r + min(rt0 + j * 16 + ln, a.r - 1)) * K + lg * 16;

  f32x4 acc[MR][RB];
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int j = 0; j < RB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  // lane group g takes elements 16 g .. 16 g + 15 of a step: 128 bytes of a
  // row per step are consecutive. K is a multiple of 8, so a piece of eight
  // is either whole or past the end.
  auto step = [&](int s, auto whole) {
    const int k = s * kStep + lg * 16;
    u32x4 xa[MR][2], ba[RB][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = decltype(whole)::value || k + 8 * h < K;
#pragma unroll
      for (int i = 0; i < MR; ++i)
        xa[i][h] = in ? *reinterpret_cast<const u32x4 *>(xp[i] + s * kStep + 8 * h) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < RB; ++j)
        ba[j][h] = in ? *reinterpret_cast<const u32x4 *>(ap[j] + s * kStep + 8 * h) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MR; ++i)
#pragma unroll
        for (int j = 0; j < RB; ++j) acc[i][j] = O::mma(xa[i][h], ba[j][h], acc[i][j]);
  };
  const int full = K / kStep, steps = (K + kStep - 1) / kStep;
  const int s0 = split * a.steps_per_split, s1 = min(s0 + a.steps_per_split, steps);
#pragma unroll 4
  for (int s = s0 + wv; s < min(s1, full); s += kWaves) step(s, std::true_type{});
  if (s1 == steps && full < steps && (full - s0) % kWaves == wv) step(full, std::false_type{});

#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int j = 0; j < RB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[wv][i * 16 + lg * 4 + q][j * 16 + ln] = acc[i][j][q];
  __syncthreads();
  for (int i = tid; i < MR * 16 * RB * 16; i += kThreads) {
    const int row = i / (RB * 16), c = i % (RB * 16);
    if (row < t.cnt && rt0 + c < a.r)
      a.part[((size_t)split * a.n + t.p0 + row) * a.r + rt0 + c] =
          (sum[0][row][c] + sum[1][row][c]) + (sum[2][row][c] + sum[3][row][c]);
  }
}

// ---- out = base + s B_a t --------------------------------------------------

__device__ inline float load_as(const void *p, size_t i, int dt) {
  if (dt == QW_DT_F32) return reinterpret_cast<const float *>(p)[i];
  const uint32_t b = reinterpret_cast<const uint16_t *>(p)[i];
  return dt == QW_DT_F16 ? Op<QW_DT_F16>::value(b) : Op<QW_DT_BF16>::value(b);
}
__device__ inline void store_as(void *p, size_t i, int dt, float v) {
  if (dt == QW_DT_F32)
    reinterpret_cast<float *>(p)[i] = v;
  else
    reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)out_bits(v, dt);
}
__device__ inline void store16(void *p, size_t i, int dt, const float (&v)[16]) {
  if (dt == QW_DT_F32) {
    f32x4 *q = reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(p) + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = f32x4{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
  } else {
    u32x4 *q = reinterpret_cast<u32x4 *>(reinterpret_cast<uint16_t *>(p) + i);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = out_bits(v[8 * k + 2 * e], dt) | (out_bits(v[8 * k + 2 * e + 1], dt) << 16);
      q[k] = w;
    }
  }
}

// A workgroup: MR x 16 rows of one adapter, cols_per_group runs of 256
// columns, 64 of each run per wave. The product is taken transposed (rows
// of B_a as the first operand), and block j of a wave's four holds the
// columns 16 g + 4 j .. + 3 of lane group g, so a lane ends with 16
// consecutive columns of one row: 16-byte loads and stores straight from
// the registers. Where N is no multiple of 8 rows start anywhere, and they
// are single elements: 4001 rows x 11008, rank 64, 78 us, x 11009 259; 64
// rows x 13824 15 us, x 13823 23. B32: base is fp32.
//
// A decode step is a chain of dependent loads (offsets, rows, then base, B
// and t), so the base and the first 64 inner elements of B are requested
// before t is put together.
template <int DT, int MR, bool B32>
__global__ __launch_bounds__(kThreads, 2) void expand_kernel(LoraArgs a) {
  using O = Op<DT>;
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];  // [2][MR * 16][ld]
  __shared__ float unit[MR * 16];  // scale times the row's power of two
  const int tid = threadIdx.x, lane = tid & 63, ln = lane & 15, lg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cg = blockIdx.x % a.col_groups;
  const RowLookup row_at(a.rows, a.n);
  const RowTile t = find_row_tile(a.offsets, a.G, a.n, MR * 16, blockIdx.x / a.col_groups, true);
  if (t.cnt == 0) return;
  const bool rest = t.g == a.G;  // rows without an adapter: base alone
  if (rest && a.in_place) return;
  const int r = a.r, rp = (r + 31) & ~31, ld = rp + 8;
  uint16_t *const hi = smem, *const lo = smem + MR * 16 * ld;

  int m[MR];
#pragma unroll
  for (int i = 0; i < MR; ++i) {
    const int q = i * 16 + ln;
    m[i] = row_at(t.p0 + min(q, t.cnt - 1));
    if (q >= t.cnt || (uint32_t)m[i] >= (uint32_t)a.n) m[i] = -1;
  }
  const bool vec = a.N % 8 == 0;  // every row starts on 16 bytes in both types

  // the loads of one column run: base, and B's first two steps of 32
  u32x4 raw[MR][B32 ? 4 : 2], w[2][4];
  const uint16_t *bp[4];
  bool in[4];
  auto request = [&](int ct) {
    const int c0 = (cg * a.cols_per_group + ct) * kColTile + wv * 64;
    const int c = c0 + lg * 16;
    if (vec && c + 16 <= a.N) {
#pragma unroll
      for (int i = 0; i < MR; ++i) {
        const size_t o = (size_t)max(m[i], 0) * a.N + c;
        const u32x4 *p = reinterpret_cast<const u32x4 *>(
            B32 ? reinterpret_cast<const char *>(reinterpret_cast<const float *>(a.base) + o)
                : reinterpret_cast<const char *>(reinterpret_cast<const uint16_t *>(a.base) + o));
#pragma unroll
        for (int k = 0; k < (B32 ? 4 : 2); ++k) raw[i][k] = p[k];
      }
    }
    if (rest) return;
    // row q of block j is column 16 (q / 4) + 4 j + q % 4
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int cb = c0 + 16 * (ln >> 2) + 4 * j + (ln & 3);
      in[j] = cb < a.N;
      bp[j] = a.B + ((size_t)t.g * a.N + (in[j] ? cb : 0)) * r + lg * 8;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        w[s][j] = s * 32 + lg * 8 < r && in[j] ? *reinterpret_cast<const u32x4 *>(bp[j] + s * 32) : u32x4{0, 0, 0, 0};
    }
  };
  request(0);

  // t of the tile: 16 lanes a row, each 8 of every 128 inner values
  if (!rest) {
    for (int row = tid >> 4; row < MR * 16; row += kThreads / 16) {
      float v[2][8];
      float top = 0.0f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int k = c * 128 + ln * 8;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[c][q] = 0.0f;
        if (row < t.cnt && k < r) {
          for (int s = 0; s < a.splits; ++s) {
            const f32x4 *p = reinterpret_cast<const f32x4 *>(a.part + ((size_t)s * a.n + t.p0 + row) * r + k);
            const f32x4 u = p[0], w = p[1];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              v[c][q] += u[q];
              v[c][q + 4] += w[q];
            }
          }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) top = fmaxf(top, fabsf(v[c][q]));
      }
#pragma unroll
      for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 16));
      // 2^-e brings top to 1..2 (within the exponents both powers have);
      // 0 and infinity stay as they are
      int e = top > 0.0f && top < INFINITY ? (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127 : 0;
      e = min(max(e, -100), 126);
      const float down = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
      if (ln == 0) unit[row] = a.scale[t.g] * __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int k = c * 128 + ln * 8;
        if (k < rp) {
          u32x4 h, l;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float f0 = v[c][2 * q] * down, f1 = v[c][2 * q + 1] * down;
            const uint32_t h0 = O::bits(f0), h1 = O::bits(f1);
            h[q] = h0 | (h1 << 16);
            l[q] = O::bits(f0 - O::value(h0)) | (O::bits(f1 - O::value(h1)) << 16);
          }
          *reinterpret_cast<u32x4 *>(hi + row * ld + k) = h;
          *reinterpret_cast<u32x4 *>(lo + row * ld + k) = l;
        }
      }
    }
    __syncthreads();
  }

  for (int ct = 0; ct < a.cols_per_group; ++ct) {
    const int c0 = (cg * a.cols_per_group + ct) * kColTile + wv * 64;
    if (c0 >= a.N) return;
    f32x4 acc[MR][4];
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    auto product = [&](int k, const u32x4 (&b)[4]) {
#pragma unroll
      for (int i = 0; i < MR; ++i) {
        const u32x4 h = *reinterpret_cast<const u32x4 *>(hi + (i * 16 + ln) * ld + k + lg * 8);
        const u32x4 l = *reinterpret_cast<const u32x4 *>(lo + (i * 16 + ln) * ld + k + lg * 8);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = O::mma(b[j], l, acc[i][j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = O::mma(b[j], h, acc[i][j]);
      }
    };
    if (!rest) {
      product(0, w[0]);
      if (rp > 32) product(32, w[1]);
      for (int k = 64; k < rp; k += 32) {
        u32x4 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          b[j] = k + lg * 8 < r && in[j] ? *reinterpret_cast<const u32x4 *>(bp[j] + k) : u32x4{0, 0, 0, 0};
        product(k, b);
      }
    }
    const int c = c0 + lg * 16;
    if (c < a.N) {
#pragma unroll
      for (int i = 0; i < MR; ++i) {
        if (m[i] < 0) continue;
        const size_t o = (size_t)m[i] * a.N + c;
        const float u = rest ? 0.0f : unit[i * 16 + ln];
        if (vec && c + 16 <= a.N) {
          float v[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            if (B32) {
              const uint32_t b32 = raw[i][q >> 2][q & 3];
              v[q] = __builtin_bit_cast(float, b32);
            } else {
              const uint32_t b16 = (raw[i][(q >> 3) & 1][(q >> 1) & 3] >> (16 * (q & 1))) & 0xFFFFu;
              v[q] = a.base_dtype == QW_DT_F16 ? Op<QW_DT_F16>::value(b16) : Op<QW_DT_BF16>::value(b16);
            }
            if (!rest) v[q] = __builtin_fmaf(u, acc[i][q >> 2][q & 3], v[q]);
          }
          store16(a.out, o, a.out_dtype, v);
        } else {
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            if (c + q < a.N) {
              float v = load_as(a.base, o + q, a.base_dtype);
              if (!rest) v = __builtin_fmaf(u, acc[i][q >> 2][q & 3], v);
              store_as(a.out, o + q, a.out_dtype, v);
            }
          }
        }
      }
    }
    if (ct + 1 < a.cols_per_group) request(ct + 1);
  }
}

// Row tiles of 64 once the adapters have some 24 rows each, so that the
// adapters are read by fewer workgroups (A x of 4001 rows, K = 4096, rank
// 64: 16 us, 20 with tiles of 32); else 16.
int row_blocks(int n, int G) { return n >= 24 * G ? 4 : 1; }

// Splits of K: enough workgroups to fill the card, of at least four steps
// (one a wave).
int k_splits(const qw_adapters *ad, int n, int *per) {
  const int steps = (ad->K + kStep - 1) / kStep;
  const int rank_tiles = (ad->r + 63) / 64;
  const long long tiles = most_row_tiles(n, ad->count, 16 * row_blocks(n, ad->count)) * rank_tiles;
  long long splits = (384 + tiles - 1) / tiles;
  if (splits > steps / 4) splits = steps / 4;
  if (splits > 16) splits = 16;
  if (splits < 1) splits = 1;
  *per = (int)((steps + splits - 1) / splits);
  return (steps + *per - 1) / *per;
}

bool adapters_ok(const qw_adapters *ad) {
  return ad && ad->count >= 1 && ad->N >= 1 && ad->K >= 8 && ad->K % 8 == 0 && ad->r >= 8 && ad->r % 8 == 0;
}

template <int DT, int MR>
qw_status launch_lora(LoraArgs a, hipStream_t s) {
  a.rank_tiles = (a.r + 63) / 64;
  const long long tiles = most_row_tiles(a.n, a.G, MR * 16);
  const long long g1 = tiles * a.rank_tiles * a.splits;
  const int col_tiles = (a.N + kColTile - 1) / kColTile;
  // the second launch takes half as many rows a workgroup: its registers
  // hold base, B and the sums, and three waves a SIMD keep more in flight
  // than two (4001 rows x 11008, rank 64: 62 us against 70)
  constexpr int ME = MR > 1 ? MR / 2 : 1;
  const long long tiles2 = most_row_tiles(a.n, a.G + 1, ME * 16);
  // several column runs per workgroup once there are three workgroups a CU,
  // so that t is read and split fewer times (64 rows x 13824 by 32 adapters:
  // 10 us; 14 both with a run per workgroup and with half as many workgroups)
  long long per = tiles2 * col_tiles / 768;
  a.cols_per_group = (int)(per < 1 ? 1 : per > 8 ? 8 : per);
  a.col_groups = (col_tiles + a.cols_per_group - 1) / a.cols_per_group;
  const long long g2 = tiles2 * a.col_groups;
  if (g1 > kMostBlocks || g2 > kMostBlocks) return QW_ERR_UNSUPPORTED;
  if (a.r <= 16)
    QW_HIP_TRY(launch(shrink_kernel<DT, MR, 1>, (unsigned)g1, kThreads, 0, s, a));
  else if (a.r <= 32)
    QW_HIP_TRY(launch(shrink_kernel<DT, MR, 2>, (unsigned)g1, kThreads, 0, s, a));
  else
    QW_HIP_TRY(launch(shrink_kernel<DT, MR, 4>, (unsigned)g1, kThreads, 0, s, a));
  static_assert(2 * ME * 16 * (QW_MAX_RANK + 8) * 2 <= 64 * 1024, "a launch needs no attribute for its LDS");
  const size_t lds = (size_t)2 * ME * 16 * (((a.r + 31) & ~31) + 8) * 2;
  const auto expand = a.base_dtype == QW_DT_F32 ? expand_kernel<DT, ME, true> : expand_kernel<DT, ME, false>;
  QW_HIP_TRY(launch(expand, (unsigned)g2, kThreads, lds, s, a));
  return QW_OK;
}

}  // namespace
}  // namespace qw

extern "C" {

size_t qw_lora_workspace_bytes(const qw_adapters *ad, int n) {
  if (!qw::adapters_ok(ad) || ad->count > QW_MAX_GROUPS || ad->r > QW_MAX_RANK || n < 1 || n > QW_MAX_ROWS) return 0;
  int per;
  return (size_t)qw::k_splits(ad, n, &per) * (size_t)n * (size_t)ad->r * sizeof(float);
}

qw_status qw_lora_add(const qw_adapters *ad, const void *x, const qw_groups *g, const void *base,
                      qw_dtype base_dtype, void *out, qw_dtype out_dtype, void *workspace,
                      size_t workspace_bytes, void *stream) {
  using namespace qw;
  CallScope scope;
  if (!adapters_ok(ad) || !ad->A || !ad->B || !ad->scale || !x || !base || !out) return QW_ERR_INVALID_ARG;
  if (ad->dtype != QW_DT_F16 && ad->dtype != QW_DT_BF16) return QW_ERR_INVALID_ARG;
  if (!is_dtype(base_dtype) || !is_dtype(out_dtype)) return QW_ERR_INVALID_ARG;
  if (base == out && base_dtype != out_dtype) return QW_ERR_INVALID_ARG;
  QW_TRY(check_groups(g));
  if (g->G != ad->count) return QW_ERR_INVALID_ARG;
  if (ad->r > QW_MAX_RANK) return QW_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < qw_lora_workspace_bytes(ad, g->n)) return QW_ERR_INVALID_ARG;
  if (!aligned16(ad->A) || !aligned16(ad->B) || !aligned16(ad->scale) || !aligned16(x) || !aligned16(base) ||
      !aligned16(out) || !aligned16(workspace))
    return QW_ERR_ALIGNMENT;
  QW_TRY(current_device(nullptr));
  LoraArgs a{};
  a.x = reinterpret_cast<const uint16_t *>(x);
  a.A = reinterpret_cast<const uint16_t *>(ad->A);
  a.B = reinterpret_cast<const uint16_t *>(ad->B);
  a.scale = ad->scale;
  a.offsets = g->offsets;
  a.rows = g->rows;
  a.base = base;
  a.out = out;
  a.part = reinterpret_cast<float *>(workspace);
  a.n = g->n;
  a.G = g->G;
  a.N = ad->N;
  a.K = ad->K;
  a.r = ad->r;
  a.splits = k_splits(ad, g->n, &a.steps_per_split);
  a.base_dtype = base_dtype;
  a.out_dtype = out_dtype;
  a.in_place = base == out;
  const bool tall = row_blocks(g->n, g->G) == 4;
  if (ad->dtype == QW_DT_F16)
    return tall ? launch_lora<QW_DT_F16, 4>(a, as_stream(stream)) : launch_lora<QW_DT_F16, 1>(a, as_stream(stream));
  return tall ? launch_lora<QW_DT_BF16, 4>(a, as_stream(stream)) : launch_lora<QW_DT_BF16, 1>(a, as_stream(stream));
}

}  // extern "C"
