// The experts' products by wide tiles, for many rows per expert:
//   Y[p][n] = sum_k X[r(p)][k] w_e[n][k],  e = group of position p
//
// What bounds it: the matrix cores, and beside them the vector units that
// scale. As in the narrow kernel the products are with bare code levels
// (exact in 16 bits: +-152, +-45 for 2-bit, 16 + u for INT4 with the sums
// started at -24 times those of x; for NF4 the 16 levels times the constant
// that rounds them best), 32 (NF4: 64) weights a
// product, and each fp32 result is scaled into the accumulator by one
// multiply-add: 16 cycles of the vector unit beside 16 of the matrix core.
// Scaling the weights instead rounds each to 16 bits (the tall tiles do).
// Measured: 12000 rows over 64 gated experts of 2816 x 2048 in INT4 298 us,
// 0.46 PFLOP/s; the matrix cores busy 0.28 of the cycles, vector
// instructions issuing in 0.63 of them (2-bit, 8192 rows of 14336 x 4096).
//
// Tile: 16 MR rows x 256 columns, by four waves of 64 columns each. X goes
// through LDS, 64 elements of K at a time, two buffers; pieces of 16 bytes
// are stored at their place xor row % 8, so that both the copies and the
// operand reads spread over the banks. Each wave loads the codes of its own
// columns, transposes them over its lane groups and reads their levels from
// the table: no weight goes through LDS twice.
//
// 2-bit: Z times the group sums of x is a product of its own with K / 32
// inner elements, taken every 32 groups: the sums come from one matrix
// product per row block and group against ones (the waves in turn), wait in
// LDS as fp32 and enter as two bf16 numbers, as the fp16 Z does.
#include <math.h>

#include <mutex>
#include <type_traits>

#include "experts.h"

namespace qw {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kSub = 4;       // 16-column blocks of a wave
constexpr int kStage = 64;    // K elements of one LDS buffer
constexpr int kSumLd = 36;    // floats per row of a window of 32 group sums

template <int FMT, int DT, bool ANCH, int MR>
__global__ __launch_bounds__(kThreads, 2) void wide_kernel(ExpertArgs a) {
  using O = Op<DT>;
  constexpr bool k2 = FMT == QW_FMT_2BIT_G32, kN = FMT == QW_FMT_NF4_B64, k4 = FMT == QW_FMT_INT4_G32;
  constexpr int kRows = 16 * MR;
  constexpr int kPieces = kRows * 8 / kThreads;  // 16-byte pieces of X per thread and stage
  constexpr int kSpan = k2 ? 256 : 128;          // weights of a column in one set of code loads
  constexpr int kPer = kSpan / kStage;           // stages of a set
  constexpr int kCodeDiv = k2 ? 4 : 2, kScaleDiv = k2 ? 8 : 16;
  static_assert(kPieces >= 1, "every thread copies a piece");

  __shared__ __attribute__((aligned(16))) char tab[k4 ? 16 : 256 * kEntry];
  // the X buffers; behind the loop the waves' slabs lie there
  constexpr int kBuf = kRows * kStage * 2, kSlabLd = kSub * 16 + 4;
  constexpr int kSlab = kWaves * 16 * kSlabLd * 4;
  __shared__ __attribute__((aligned(16))) char xs[2 * kBuf > kSlab ? 2 * kBuf : kSlab];
  __shared__ __attribute__((aligned(16))) float sums[k2 ? 2 : 1][k2 ? kRows : 1][kSumLd];

  const int tid = threadIdx.x, lane = tid & 63, ln = lane & 15, lg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = a.K, stages = K / kStage;

  const TileAt at = place_tile(a.offsets, a.G, a.n, kRows, a.col_tiles, (int)blockIdx.x);
  if (at.rows.cnt == 0) return;
  const RowTile rt = at.rows;
  const int e = rt.g;
  if (!k4) fill_table<FMT, DT, kThreads, true>(tab, a);

  // ---- X: this thread's pieces; rows past the tile repeat its first row ----
  const int pc = tid & 7, pr = tid >> 3;
  const uint16_t *xp[kPieces];
  uint32_t xat[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int row = pr + 32 * i;
    const int p = rt.p0 + (row < rt.cnt ? row : 0);
    const int xr = a.x_div ? max(x_row(a.rows[p], a.x_div, a.x_rows), 0) : p;
    xp[i] = a.X + (size_t)xr * K + pc * 8;
    xat[i] = (uint32_t)row * (kStage * 2) + (uint32_t)((pc ^ (row & 7)) * 16);
  }
  u32x4 xv[kPieces];
  uint32_t drop = 0;  // anchor bits of this thread's eight channels
  // stages past the end copy zeros
  uint32_t live = 0;
  auto load_x = [&](int st) {
    const int at = min(st, stages - 1);
    live = st < stages ? 0xFFFFFFFFu : 0u;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) xv[i] = *reinterpret_cast<const u32x4 *>(xp[i] + at * kStage);
    if (k2 && ANCH) drop = a.mask[(size_t)e * (K / 32) + at * 2 + (pc >> 2)] >> (8 * (pc & 3));
  };
  auto store_x = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      u32x4 v = xv[i];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t keep = live;
        if (k2 && ANCH) keep &= ~(((drop >> (2 * q)) & 1 ? 0xFFFFu : 0u) | ((drop >> (2 * q + 1)) & 1 ? 0xFFFF0000u : 0u));
        v[q] &= keep;
      }
      if (k4) v = Int4<DT>::order(v);
      *reinterpret_cast<u32x4 *>(xs + buf * kBuf + xat[i]) = v;
    }
  };
  // operand of row block i, 32-weight step h of the buffer
  const uint32_t xrd = (uint32_t)ln * (kStage * 2);
  auto read_a = [&](int buf, int i, int h) {
    return *reinterpret_cast<const u32x4 *>(xs + buf * kBuf + i * 16 * kStage * 2 + xrd + (((h * 4 + lg) ^ (ln & 7)) * 16));
  };

  // ---- W: this lane's column in each of the wave's four blocks ----
  const int half_cols = a.swiglu ? 32 : 64;  // output columns of a wave
  const int c0 = at.col * (half_cols * kWaves) + wv * half_cols;
  const size_t cb = (size_t)a.N * (K / kCodeDiv), sb = (size_t)a.N * (K / kScaleDiv);
  const auto rc = rsrc(a.codes + (size_t)e * cb, (uint32_t)cb);
  const auto rs = rsrc(a.scales + (size_t)e * sb, (uint32_t)sb);
  int wn[kSub];
#pragma unroll
  for (int j = 0; j < kSub; ++j) {
    const int h = c0 + (a.swiglu ? (j & 1) : j) * 16 + ln;
    wn[j] = h < a.out_n ? (a.swiglu ? h + (j >> 1) * a.out_n : h) : -1;
  }
  // codes and scale words of one set; lane group g holds the g-th quarter.
  // scale words: 2-bit two groups of (S, Z); INT4 one fp16; NF4 the absmax
  // of the block of 64 that holds the quarter
  struct Set {
    u32x4 c[kSub];
    uint32_t s[kSub][k2 ? 2 : 1];
  };
  auto load_w = [&](int set, Set &d) {
    const int k = set * kSpan + lg * (kSpan / 4);
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      const bool in = k < K && wn[j] >= 0;
      const uint32_t oc = in ? (uint32_t)wn[j] * (uint32_t)(K / kCodeDiv) + (uint32_t)k / kCodeDiv : kOob;
      const uint32_t os = in ? (uint32_t)wn[j] * (uint32_t)(K / kScaleDiv) + (uint32_t)(kN ? k & ~63 : k) / kScaleDiv : kOob;
      d.c[j] = __builtin_amdgcn_raw_buffer_load_b128(rc, (int)oc, 0, 0);
      if (k2) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rs, (int)os, 0, 0);
        d.s[j][0] = v[0];
        d.s[j][k2 ? 1 : 0] = v[1];
      } else if (kN) {
        d.s[j][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)os, 0, 0);
      } else {
        d.s[j][0] = __builtin_amdgcn_raw_buffer_load_b16(rs, (int)os, 0, 0);
      }
    }
  };
  auto arrange = [&](Set &d) {
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      uint32_t w[4] = {d.c[j][0], d.c[j][1], d.c[j][2], d.c[j][3]};
      if (k2) to_halves(w);
      transpose4(w);
      d.c[j] = u32x4{w[0], w[1], w[2], w[3]};
    }
  };
  const uint32_t rep = k2 ? (uint32_t)(lane & 15) * 8u : (uint32_t)(lane & 31) * 4u;
  uint32_t sixteen = Int4<DT>::kSixteen;
  if (k4) asm volatile("" : "+v"(sixteen));  // an and-or takes one scalar operand
  // operand of column block j for step h of stage s of the set
  auto make_b = [&](const Set &d, int j, int s, int h) {
    if (k2) {
      const uint32_t c = d.c[j][s] >> (16 * h);
      const u32x2 lo = *reinterpret_cast<const u32x2 *>(tab + (((c & 0xFFu) << 7) | rep));
      const u32x2 hi = *reinterpret_cast<const u32x2 *>(tab + ((((c >> 8) & 0xFFu) << 7) | rep));
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
    const uint32_t c = d.c[j][2 * (s & 1) + h];
    if (k4) return Int4<DT>::operand(c, sixteen);
    u32x4 b;
#pragma unroll
    for (int q = 0; q < 4; ++q) b[q] = *reinterpret_cast<const uint32_t *>(tab + ((((c >> (8 * q)) & 0xFFu) << 7) | rep));
    return b;
  };
  // the scale of block j in step h of stage s, to all lane groups
  auto scale_of = [&](const Set &d, int j, int s, int h) {
    if (k2) return f16_bits_to_f32((uint16_t)from_group(d.s[j][h], s));
    if (kN) return __builtin_bit_cast(float, from_group(d.s[j][0], 2 * s + h)) * a.level_unit;
    return f16_bits_to_f32((uint16_t)from_group(d.s[j][0], 2 * s + h));
  };

  f32x4 acc[MR][kSub];
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int j = 0; j < kSub; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const f32x4 zero = {0, 0, 0, 0};

  // products of one stage out of buffer buf. The results of one row block
  // are scaled while those of the next are computed; the scheduling barriers
  // keep the compiler from starting all of them first, which costs more
  // registers than two waves a SIMD have.
  auto multiply = [&](int st, int buf, const Set &d, int s) {
    constexpr int kHalves = kN ? 1 : 2;  // NF4: both steps share a scale
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      u32x4 b[kN ? 2 : 1][kSub];
      float sc[kSub];
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        b[0][j] = make_b(d, j, s, h);
        if (kN) b[kN ? 1 : 0][j] = make_b(d, j, s, 1);
        sc[j] = scale_of(d, j, s, h);
      }
      if (k2) {  // the group's sums of x: row block wv (and wv + 4) is this wave's
        const uint32_t one = O::bits(1.0f) * 0x10001u;
        const int group = 2 * st + h;
#pragma unroll
        for (int i0 = 0; i0 < MR; i0 += kWaves) {
          const int i = i0 + (MR < kWaves ? wv % MR : wv);  // fewer blocks than waves: twice the same
          const f32x4 g = O::mma(read_a(buf, i, h), u32x4{one, one, one, one}, zero);
          // every column holds the same four rows' sums: column c writes row c % 4
          const float v = ln & 2 ? (ln & 1 ? g[3] : g[2]) : (ln & 1 ? g[1] : g[0]);
          sums[k2 ? (group >> 5) & 1 : 0][k2 ? i * 16 + lg * 4 + (ln & 3) : 0][group & 31] = v;
        }
      }
      f32x4 dd[2][kSub];
#pragma unroll
      for (int i = 0; i <= MR; ++i) {
        if (i < MR) {
          const u32x4 x = read_a(buf, i, h);
          u32x4 x1;
          if (kN) x1 = read_a(buf, i, 1);
          constexpr uint32_t m24 = Int4<DT>::kMinus24;
          const f32x4 start = k4 ? O::mma(x, u32x4{m24, m24, m24, m24}, zero) : zero;
#pragma unroll
          for (int j = 0; j < kSub; ++j) {
            f32x4 &t = dd[i & 1][j];
            t = O::mma(x, b[0][j], start);
            if (kN) t = O::mma(x1, b[kN ? 1 : 0][j], t);
          }
        }
        if (i > 0) {
#pragma unroll
          for (int j = 0; j < kSub; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i - 1][j][r] = __builtin_fmaf(sc[j], dd[(i - 1) & 1][j][r], acc[i - 1][j][r]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // the sums are due here: nothing of the scaling moves behind a branch
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
      for (int j = 0; j < kSub; ++j) asm volatile("" : "+v"(acc[i][j]));
  };

  // 2-bit: Z times the sums of the window of 32 groups from g0 on. The
  // levels are a hundredfold, so Z is too: 100 on the sums.
  auto add_offsets = [&](int g0) {
    using F = Op<QW_DT_BF16>;
    int el = lane;
    asm volatile("" : "+v"(el));
    const int groups = K / 32, g = g0 + (el >> 4) * 8;
    u32x4 zh[kSub], zl[kSub];
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      uint32_t w[8];
#pragma unroll
      for (int q = 0; q < 8; q += 2) {  // two groups a load: K is a multiple of 64
        const bool in = g + q < groups && wn[j] >= 0;
        const uint32_t o = in ? (uint32_t)wn[j] * (uint32_t)(K / kScaleDiv) + (uint32_t)(g + q) * 4u : kOob;
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rs, (int)o, 0, 0);
        w[q] = v[0];
        w[q + 1] = v[1];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float z0 = f16_bits_to_f32((uint16_t)(w[2 * q] >> 16)), z1 = f16_bits_to_f32((uint16_t)(w[2 * q + 1] >> 16));
        const uint32_t h0 = F::bits(z0), h1 = F::bits(z1);
        zh[j][q] = h0 | (h1 << 16);
        zl[j][q] = F::bits(z0 - F::value(h0)) | (F::bits(z1 - F::value(h1)) << 16);
      }
    }
#pragma unroll
    for (int i = 0; i < MR; ++i) {
      const float *sp = &sums[k2 ? (g0 >> 5) & 1 : 0][k2 ? i * 16 + (el & 15) : 0][(el >> 4) * 8];
      u32x4 xh, xl;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float s0 = g + 2 * q < groups ? sp[2 * q] * 100.0f : 0.0f;
        const float s1 = g + 2 * q + 1 < groups ? sp[2 * q + 1] * 100.0f : 0.0f;
        const uint32_t h0 = F::bits(s0), h1 = F::bits(s1);
        xh[q] = h0 | (h1 << 16);
        xl[q] = F::bits(s0 - F::value(h0)) | (F::bits(s1 - F::value(h1)) << 16);
      }
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        acc[i][j] = F::mma(xl, zh[j], acc[i][j]);
        acc[i][j] = F::mma(xh, zl[j], acc[i][j]);
        acc[i][j] = F::mma(xh, zh[j], acc[i][j]);
      }
    }
  };

  // ---- the loop over K ----
  Set cur, next;
  load_w(0, next);
  load_x(0);
  store_x(0);
  __syncthreads();  // the level table too
  // (a last set that K fills in part is multiplied whole, against zeros: a
  // condition around the products makes the compiler copy the accumulators)
  const int sets = (stages + kPer - 1) / kPer;
  for (int set = 0; set < sets; ++set) {
    cur = next;
    arrange(cur);
    load_w(set + 1, next);  // past the end: zeros
#pragma unroll
    for (int s = 0; s < kPer; ++s) {
      const int st = set * kPer + s;
      load_x(st + 1);
      multiply(st, s & 1, cur, s);
      store_x((s + 1) & 1);
      __syncthreads();
    }
    if (k2 && ((set & 3) == 3 || set == sets - 1)) add_offsets((set & ~3) * 8);
  }
  if (k2) {
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
      for (int j = 0; j < kSub; ++j) acc[i][j] *= 0.01f;
  }

  // ---- anchors: 64 channels a stage, their x gathered into the buffers ----
  if (ANCH) {
    for (int o0 = 0; o0 < a.n_out; o0 += kStage) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        u32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int o = o0 + pc * 8 + q;
          if (o < a.n_out) {
            int k = o;
            if (k2) {
              k = a.idx[(size_t)e * a.n_out + o];
              if ((uint32_t)k >= (uint32_t)K) k = 0;
            }
            v[q >> 1] |= (uint32_t)xp[i][k - pc * 8] << (16 * (q & 1));
          }
        }
        *reinterpret_cast<u32x4 *>(xs + xat[i]) = v;
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int o = o0 + h * 32 + lg * 8;
        u32x4 b[kSub], b2[kSub];
#pragma unroll
        for (int j = 0; j < kSub; ++j) {
          b[j] = b2[j] = u32x4{0, 0, 0, 0};
          if (wn[j] >= 0 && o < a.n_out_pad) {
            b[j] = *reinterpret_cast<const u32x4 *>(a.wo + ((size_t)e * a.N + wn[j]) * a.n_out_pad + o);
            if (DT == QW_DT_BF16) split_f16(b[j], b2[j]);
          }
        }
#pragma unroll
        for (int i = 0; i < MR; ++i) {
          const u32x4 x = read_a(0, i, h);
#pragma unroll
          for (int j = 0; j < kSub; ++j) {
            acc[i][j] = O::mma(x, b[j], acc[i][j]);
            if (DT == QW_DT_BF16) acc[i][j] = O::mma(x, b2[j], acc[i][j]);
          }
        }
      }
      __syncthreads();
    }
  }

  // ---- epilogue: one row block at a time through the wave's slab, from
  //      column-per-lane to 16 (gated: 8) consecutive columns of a row ----
  float(*const slab)[kSlabLd] = reinterpret_cast<float(*)[kSlabLd]>(xs + wv * 16 * kSlabLd * 4);
  // (lane numbers from copies the compiler cannot see through, here and in
  // add_offsets, so that no address of theirs is computed before the loop
  // and held in registers through it)
  int el = lane;
  asm volatile("" : "+v"(el));
  const int eln = el & 15, elg = el >> 4;
  const int row = el >> 2, cq = (el & 3) * (half_cols / 4);
  const bool vec = a.out_n % 8 == 0;
#pragma unroll
  for (int i = 0; i < MR; ++i) {
#pragma unroll
    for (int j = 0; j < kSub; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) slab[elg * 4 + r][j * 16 + eln] = acc[i][j][r];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    const int rr = i * 16 + row;
    int yr = -1;
    if (rr < rt.cnt) {
      yr = rt.p0 + rr;
      if (a.by_slot) {
        yr = a.rows[yr];
        if ((uint32_t)yr >= (uint32_t)a.n) yr = -1;
      } else if (a.x_div && x_row(a.rows[yr], a.x_div, a.x_rows) < 0) {
        yr = -1;
      }
    }
#pragma unroll
    for (int q = 0; q < 16; q += 8) {
      if (q >= half_cols / 4 || yr < 0 || c0 + cq + q >= a.out_n) continue;
      float v[8];
#pragma unroll
      for (int t = 0; t < 8; t += 4) {
        const f32x4 w = *reinterpret_cast<const f32x4 *>(&slab[row][cq + q + t]);
        v[t] = w[0]; v[t + 1] = w[1]; v[t + 2] = w[2]; v[t + 3] = w[3];
      }
      if (a.swiglu) {
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = v[t] / (1.0f + expf(-v[t])) * slab[row][32 + cq + q + t];
      }
      const int n = c0 + cq + q;
      const size_t o = (size_t)yr * a.out_n + n;
      if (vec) {  // then the eight columns are all inside
        if (a.y_dtype == QW_DT_F32) {
          f32x4 *y = reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(a.Y) + o);
          y[0] = f32x4{v[0], v[1], v[2], v[3]};
          y[1] = f32x4{v[4], v[5], v[6], v[7]};
        } else {
          u32x4 w;
#pragma unroll
          for (int t = 0; t < 4; ++t) w[t] = out_bits(v[2 * t], a.y_dtype) | (out_bits(v[2 * t + 1], a.y_dtype) << 16);
          *reinterpret_cast<u32x4 *>(reinterpret_cast<uint16_t *>(a.Y) + o) = w;
        }
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          if (n + t >= a.out_n) continue;
          if (a.y_dtype == QW_DT_F32)
            reinterpret_cast<float *>(a.Y)[o + t] = v[t];
          else
            reinterpret_cast<uint16_t *>(a.Y)[o + t] = (uint16_t)out_bits(v[t], a.y_dtype);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  }
}

// The factor in 1..2 that leaves the 16 NF4 levels, times it, closest to
// numbers of the given significand bits (smallest sum of squared relative
// errors over 4096 candidates).
double best_level_factor(int bits) {
  const float *L = nf4_levels_host();
  double best = 1.0, least = 1e300;
  for (int i = 0; i < 4096; ++i) {
    const double f = 1.0 + i / 4096.0;
    double sum = 0.0;
    for (int q = 0; q < 16; ++q) {
      const double v = fabs((double)L[q]) * f;
      if (v == 0.0) continue;
      int ex;
      const double m = ldexp(frexp(v, &ex), bits);
      const double d = (rint(m) - m) / m;
      sum += d * d;
    }
    if (sum < least) {
      least = sum;
      best = f;
    }
  }
  return best;
}

template <int FMT, int DT, bool ANCH, int MR>
qw_status launch_one(const ExpertArgs &a, hipStream_t s) {
  const long long grid = most_row_tiles(a.n, a.G, 16 * MR) * a.col_tiles;
  if (grid > kMostBlocks) return QW_ERR_UNSUPPORTED;
  QW_HIP_TRY(launch(wide_kernel<FMT, DT, ANCH, MR>, (unsigned)grid, kThreads, 0, s, a));
  return QW_OK;
}

template <int FMT, int DT, bool ANCH>
qw_status launch_rows(int row_blocks, const ExpertArgs &a, hipStream_t s) {
  return row_blocks <= 2 ? launch_one<FMT, DT, ANCH, 2>(a, s) : launch_one<FMT, DT, ANCH, 4>(a, s);
}

template <int DT>
qw_status launch_fmt(int fmt, int row_blocks, const ExpertArgs &a, hipStream_t s) {
  if (fmt == QW_FMT_2BIT_G32)
    return a.n_out ? launch_rows<QW_FMT_2BIT_G32, DT, true>(row_blocks, a, s)
                   : launch_rows<QW_FMT_2BIT_G32, DT, false>(row_blocks, a, s);
  if (fmt == QW_FMT_INT4_G32)
    return a.n_out ? launch_rows<QW_FMT_INT4_G32, DT, true>(row_blocks, a, s)
                   : launch_rows<QW_FMT_INT4_G32, DT, false>(row_blocks, a, s);
  return launch_rows<QW_FMT_NF4_B64, DT, false>(row_blocks, a, s);
}

}  // namespace

qw_status launch_experts_wide(int fmt, int x_dtype, int row_blocks, const ExpertArgs &args, hipStream_t s) {
  ExpertArgs a = args;
  const int cols = kWaves * (a.swiglu ? 32 : 64);
  a.col_tiles = (a.out_n + cols - 1) / cols;
  if (fmt == QW_FMT_NF4_B64) {
    static std::once_flag once;
    static double factor[2];
    std::call_once(once, [] {
      factor[0] = best_level_factor(11);
      factor[1] = best_level_factor(8);
    });
    const double f = factor[x_dtype == QW_DT_BF16];
    for (int i = 0; i < 16; ++i) a.nf4[i] = (float)(a.nf4[i] * f);
    a.level_unit = (float)(1.0 / f);
  }
  return x_dtype == QW_DT_F16 ? launch_fmt<QW_DT_F16>(fmt, row_blocks, a, s)
                              : launch_fmt<QW_DT_BF16>(fmt, row_blocks, a, s);
}

}  // namespace qw
