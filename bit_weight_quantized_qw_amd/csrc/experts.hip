// Products of grouped rows with the packed weights of their experts, for
// few rows per expert, and the weighted sum of a token's experts.
//
//   Y[p][n] = sum_k X[r(p)][k] w_e[n][k],  e = group of position p
//
// What bounds it: a decode step reads the packed weights of every expert
// that some row takes, once, and little else; so the kernel is built to
// stream codes, and the decoding of a weight is kept to a few integer
// operations on lanes that the loads leave idle.
//
// Tile: 16 rows of one expert times 64 of its output columns, by a
// workgroup of four waves that each take a quarter of K (their fp32 sums
// are added in wave order through LDS). One v_mfma_f32_16x16x32 covers 16
// rows, 16 columns and the 32 weights of one scale group, so the products
// are with the bare code levels and the group's scale multiplies the fp32
// sum: no weight is rounded to 16 bits, and the scaling costs four
// multiply-adds a lane where scaling the weights would cost eight.
//   2-bit: the levels +-1.52, +-0.45 enter as +-152, +-45 (exact in fp16
//     and bf16), the sum is divided by 100 at the end; Z times the row sums
//     of x, which come from the same A operand against a constant 100.
//   INT4: 16 + u, made from the nibbles without a table, the products
//     starting from -24 times the row sums of x. NF4: a level is two 16-bit
//     numbers, the nearest and the rest, two products.
// A code byte of the other formats becomes 16-bit levels by one LDS table
// read. Lane l reads replica l % 16 of the table, so no two of 16 lanes meet
// in a bank. Up to four rows, four scale groups share one result (below).
//
// Measured: 40 tokens, 2 of 16 experts of 8192 x 4096, in NF4 73 to 88 us
// (3.4 to 4.2 TB/s), in 2-bit 69 us (2.9 TB/s; INT4 takes wide tiles of 32
// rows there, 92 us); 136 slots over 64 experts of 2048 x 1408 in 2-bit with
// anchors 29 us, 2.7 TB/s; one token's 8 of 64 experts of 2816 x 2048 12 us,
// of which 9 are one workgroup: 1 until its tile is known, 4 until its first
// codes are there, 1.3 a chunk of 256 weights, 0.5 for the sums.
//
// A lane loads 64 consecutive codes of one column (16 bytes of 2-bit, 32 of
// 4-bit codes); the matrix instruction wants eight per lane of 32
// consecutive ones. A 4 x 4 transposition of dwords over the four lane
// groups (two half-wave and two row swaps) turns one into the other.
#include <math.h>

#include <type_traits>

#include "experts.h"

namespace qw {
namespace {

constexpr int kRows = 16;
constexpr int kCols = 64;
constexpr int kSub = kCols / 16;  // 16-column blocks of a tile
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kChunk = 256;       // weights of one column in one set of loads

// The tile's gathered loads of one chunk: codes and scale words of the
// lane's 64 weights in each of the four 16-column blocks.
template <int FMT>
struct Chunk {
  static constexpr int kCodes = FMT == QW_FMT_2BIT_G32 ? 4 : 8;   // dwords
  static constexpr int kScales = FMT == QW_FMT_2BIT_G32 ? 2 : 1;  // dwords
  uint32_t c[kSub][kCodes];
  uint32_t s[kSub][kScales];
};

template <int FMT, int DT, bool ANCH>
__global__ __launch_bounds__(kThreads, 3) void experts_kernel(ExpertArgs a) {
  using O = Op<DT>;
  // the level table; behind the loop the waves' sums lie there
  constexpr bool k4 = FMT == QW_FMT_INT4_G32;
  constexpr int kSums = kWaves * kRows * (kCols + 4) * 4, kTable = k4 ? 0 : 256 * kEntry;
  __shared__ __attribute__((aligned(16))) char tab[kTable > kSums ? kTable : kSums];
  float(*const part)[kRows][kCols + 4] = reinterpret_cast<float(*)[kRows][kCols + 4]>(tab);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, lg = lane >> 4;
  const int tile = blockIdx.x / a.col_tiles, ct = blockIdx.x % a.col_tiles;
  const RowLookup row_at(a.rows, a.n);
  const RowTile rt = find_row_tile(a.offsets, a.G, a.n, kRows, tile);
  if (rt.cnt == 0) return;
  const int e = rt.g, K = a.K;

  // this lane's row of A: rows past the tile's end repeat its first row
  // (their products are not stored)
  const bool few = rt.cnt <= 4;
  const int lr = few ? ln & 3 : ln;
  const int p = rt.p0 + (lr < rt.cnt ? lr : 0);
  int xr = a.x_div ? row_at(p) : p;

  // columns: gated tiles take 32 gate columns and the same 32 up columns
  const int half_cols = a.swiglu ? kCols / 2 : kCols;
  const int c0 = ct * half_cols;
  uint32_t co[kSub], so[kSub];
  constexpr int kCodeDiv = FMT == QW_FMT_2BIT_G32 ? 4 : 2;     // weights per code byte
  constexpr int kScaleDiv = FMT == QW_FMT_2BIT_G32 ? 8 : 16;   // weights per scale byte
  const size_t cb = (size_t)a.N * (K / kCodeDiv), sb = (size_t)a.N * (K / kScaleDiv);
  const auto rc = rsrc(a.codes + (size_t)e * cb, (uint32_t)cb);
  const auto rs = rsrc(a.scales + (size_t)e * sb, (uint32_t)sb);
  int wn[kSub];
#pragma unroll
  for (int j = 0; j < kSub; ++j) {
    int n = c0 + j * 16 + ln;
    bool in = n < a.out_n;
    if (a.swiglu) {
      const int h = c0 + (j & 1) * 16 + ln;
      in = h < a.out_n;
      n = h + (j >> 1) * a.out_n;
    }
    wn[j] = in ? n : -1;
    co[j] = in ? (uint32_t)n * (uint32_t)(K / kCodeDiv) : kOob;
    so[j] = in ? (uint32_t)n * (uint32_t)(K / kScaleDiv) : kOob;
  }

  // this wave's chunks
  const int chunks = (K + kChunk - 1) / kChunk;
  const int per = (chunks + kWaves - 1) / kWaves;
  const int ch0 = min(wv * per, chunks), ch1 = min(ch0 + per, chunks);

  using CH = Chunk<FMT>;
  auto load = [&](int ch, CH &d) {
    const int k = ch * kChunk + lg * 64;
    const bool in = k < K;
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      const uint32_t oc = in && wn[j] >= 0 ? co[j] + (uint32_t)k / kCodeDiv : kOob;
      const uint32_t os = in && wn[j] >= 0 ? so[j] + (uint32_t)k / kScaleDiv : kOob;
#pragma unroll
      for (int i = 0; i < CH::kCodes; i += 4) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rc, (int)(oc == kOob ? kOob : oc + 4 * i), 0, 0);
        d.c[j][i] = v[0]; d.c[j][i + 1] = v[1]; d.c[j][i + 2] = v[2]; d.c[j][i + 3] = v[3];
      }
      if (few && FMT != QW_FMT_NF4_B64) {  // those of groups lg and 4 + lg of the chunk
        constexpr uint32_t kWord = FMT == QW_FMT_2BIT_G32 ? 4 : 2;
        const int g = ch * (kChunk / 32) + lg;
        const uint32_t o0 = wn[j] >= 0 && g < K / 32 ? so[j] + (uint32_t)g * kWord : kOob;
        const uint32_t o1 = wn[j] >= 0 && g + 4 < K / 32 ? so[j] + (uint32_t)(g + 4) * kWord : kOob;
        if (FMT == QW_FMT_2BIT_G32) {
          d.s[j][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)o0, 0, 0);
          d.s[j][CH::kScales - 1] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)o1, 0, 0);
        } else {
          d.s[j][0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(rs, (int)o0, 0, 0) |
                      (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(rs, (int)o1, 0, 0) << 16;
        }
      } else if (CH::kScales == 2) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rs, (int)os, 0, 0);
        d.s[j][0] = v[0];
        d.s[j][CH::kScales - 1] = v[1];
      } else {
        d.s[j][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)os, 0, 0);
      }
    }
  };

  const uint16_t *xp = a.X;  // this lane's row, once its number is there
  f32x4 acc[kSub];
#pragma unroll
  for (int j = 0; j < kSub; ++j) acc[j] = f32x4{0, 0, 0, 0};
  const f32x4 zero = {0, 0, 0, 0};
  const uint32_t rep = (uint32_t)(lane & 15) * 8u;
  uint32_t sixteen = Int4<DT>::kSixteen;
  if (k4) asm volatile("" : "+v"(sixteen));  // an and-or takes one scalar operand
  auto entry = [&](uint32_t byte) { return tab + ((byte << 7) | rep); };
  // 64 elements of X from k on: this lane's eight of each 32
  auto load_x = [&](int k, u32x4 (&d)[2]) {
    d[0] = *reinterpret_cast<const u32x4 *>(xp + k + lg * 8);
    d[1] = *reinterpret_cast<const u32x4 *>(xp + k + 32 + lg * 8);
  };

  // Operand of column block j for step h (32 weights) of run s of a chunk.
  struct Operand {
    u32x4 b, rest;  // NF4: the levels' second parts
  };
  auto operand = [&](const uint32_t (&c)[kSub][CH::kCodes], int j, int s, int h) {
    Operand o;
    if (FMT == QW_FMT_2BIT_G32) {
      const uint32_t w = c[j][s] >> (16 * h);
      const u32x2 lo = *reinterpret_cast<const u32x2 *>(entry(w & 0xFFu));
      const u32x2 hi = *reinterpret_cast<const u32x2 *>(entry((w >> 8) & 0xFFu));
      o.b = u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else if (k4) {
      o.b = Int4<DT>::operand(c[j][(4 * h + s) % CH::kCodes], sixteen);
    } else {
      const uint32_t w = c[j][(4 * h + s) % CH::kCodes];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const u32x2 l = *reinterpret_cast<const u32x2 *>(entry((w >> (8 * q)) & 0xFFu));
        o.b[q] = l[0];
        o.rest[q] = l[1];
      }
    }
    return o;
  };
  // Operand of X for the 32 elements from k on, and what goes with it: 100
  // times its row sums (2-bit, for Z) or -24 times them (INT4: the products
  // start there, so that 16 + u counts as u - 8).
  auto prepare = [&](int k, u32x4 A, u32x4 &x_op, const f32x4 &from, f32x4 &sums) {
    if (FMT == QW_FMT_2BIT_G32) {
      if (ANCH) {
        const uint32_t m = a.mask[(size_t)e * (K / 32) + k / 32] >> (8 * lg);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          A[q] &= ~(((m >> (2 * q)) & 1 ? 0xFFFFu : 0u) | ((m >> (2 * q + 1)) & 1 ? 0xFFFF0000u : 0u));
      }
      const uint32_t hundred = Op<DT>::bits(100.0f) * 0x10001u;
      sums = O::mma(A, u32x4{hundred, hundred, hundred, hundred}, from);
    }
    if (k4) {
      A = Int4<DT>::order(A);
      constexpr uint32_t m = Int4<DT>::kMinus24;
      sums = O::mma(A, u32x4{m, m, m, m}, from);
    }
    x_op = A;
  };
  // to += the products D (and sums) by the scale word w
  auto scale_in = [&](f32x4 &to, uint32_t w, const f32x4 &D, const f32x4 &sums) {
    const float S = FMT == QW_FMT_NF4_B64 ? __builtin_bit_cast(float, w) : f16_bits_to_f32((uint16_t)w);
    const float Z = f16_bits_to_f32((uint16_t)(w >> 16));
#pragma unroll
    for (int r = 0; r < 4; ++r)
      to[r] = __builtin_fmaf(S, D[r], FMT == QW_FMT_2BIT_G32 ? __builtin_fmaf(Z, sums[r], to[r]) : to[r]);
  };

  // the table while the first codes and the rows' numbers are on their way
  auto table_and_rows = [&] {
    if (!k4) {
      fill_table<FMT, DT, kThreads>(tab, a);
      __syncthreads();
    }
    if (a.x_div) xr = max(x_row(xr, a.x_div, a.x_rows), 0);
    xp = a.X + (size_t)xr * K;
  };

  // The loops over chunks stay rolled: a short launch spends much of its time
  // fetching instructions.
  if (few) {
    // Up to four rows: operand row 4 s + m is row m of X in the s-th of four
    // consecutive scale groups and zero in the others, so four products run
    // into one result, whose rows lane group s holds for its own group: one
    // scaling per four products, by a scale word that only that lane group
    // needs. The groups' sums are added up with the waves'.
    constexpr int kGroup = FMT == QW_FMT_NF4_B64 ? 64 : 32, kQuads = kChunk / (4 * kGroup);
    const int slot = ln >> 2;
    auto load_xf = [&](int ch, u32x4 (&v)[2]) {  // the lane's own groups, 16 bytes each
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int k = FMT == QW_FMT_NF4_B64 ? ch * kChunk + slot * 64 + q * 32 : ch * kChunk + (q * 4 + slot) * 32;
        v[q] = *reinterpret_cast<const u32x4 *>(xp + (k < K ? k + lg * 8 : 0));
        if (k >= K) v[q] = u32x4{0, 0, 0, 0};
      }
    };
    CH next;
    u32x4 xn[2];
    if (ch0 < ch1) load(ch0, next);
    table_and_rows();
    if (ch0 < ch1) load_xf(ch0, xn);
#pragma unroll 1
    for (int ch = ch0; ch < ch1; ++ch) {
      CH d = next;
      u32x4 x[2] = {xn[0], xn[1]};
      if (ch + 1 < ch1) {
        load(ch + 1, next);
        load_xf(ch + 1, xn);
      }
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        if (FMT == QW_FMT_2BIT_G32) to_halves(reinterpret_cast<uint32_t(&)[4]>(d.c[j][0]));
#pragma unroll
        for (int i = 0; i < CH::kCodes; i += 4) transpose4(reinterpret_cast<uint32_t(&)[4]>(d.c[j][i]));
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (FMT == QW_FMT_2BIT_G32 && ANCH) {
          const int g = ch * (kChunk / 32) + q * 4 + slot;
          const uint32_t m = g < K / 32 ? a.mask[(size_t)e * (K / 32) + g] >> (8 * lg) : 0u;
#pragma unroll
          for (int t = 0; t < 4; ++t)
            x[q][t] &= ~(((m >> (2 * t)) & 1 ? 0xFFFFu : 0u) | ((m >> (2 * t + 1)) & 1 ? 0xFFFF0000u : 0u));
        }
        if (k4) x[q] = Int4<DT>::order(x[q]);
      }
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        f32x4 sums = zero, D[kSub];
#pragma unroll
        for (int j = 0; j < kSub; ++j) D[j] = zero;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
          for (int h = 0; h < (kQuads == 1 ? 2 : 1); ++h) {
            u32x4 A = kQuads == 1 ? x[h] : x[q];
#pragma unroll
            for (int t = 0; t < 4; ++t) A[t] = slot == s ? A[t] : 0u;
            constexpr uint32_t m24 = Int4<DT>::kMinus24;
            const uint32_t hundred = Op<DT>::bits(100.0f) * 0x10001u, ones = k4 ? m24 : hundred;
            if (kQuads != 1) sums = O::mma(A, u32x4{ones, ones, ones, ones}, sums);
            // step (32 weights) 4 q + s of the chunk; NF4: 2 s + h
            const int step = kQuads == 1 ? 2 * s + h : 4 * q + s;
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
              const Operand w = operand(d.c, j, step >> 1, step & 1);
              D[j] = O::mma(A, w.b, D[j]);
              if (FMT == QW_FMT_NF4_B64) D[j] = O::mma(A, w.rest, D[j]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kSub; ++j) {
          if (k4) D[j] += sums;
          scale_in(acc[j], k4 ? d.s[j][0] >> (16 * q) : d.s[j][q % CH::kScales], D[j], sums);
        }
      }
    }
  } else {
  CH next;
  u32x4 x[4][2];
  const int k_end = min(ch1 * kChunk, K);
  if (ch0 < ch1) load(ch0, next);
  table_and_rows();
  if (ch0 < ch1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) load_x(min(ch0 * kChunk + 64 * i, k_end - 64), x[i]);
  }
#pragma unroll 1
  for (int ch = ch0; ch < ch1; ++ch) {
    CH d = next;
    if (ch + 1 < ch1) load(ch + 1, next);
    uint32_t sc[kSub][CH::kScales][4];
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      if (FMT == QW_FMT_2BIT_G32) to_halves(reinterpret_cast<uint32_t(&)[4]>(d.c[j][0]));
#pragma unroll
      for (int i = 0; i < CH::kCodes; i += 4) transpose4(reinterpret_cast<uint32_t(&)[4]>(d.c[j][i]));
#pragma unroll
      for (int i = 0; i < CH::kScales; ++i) gather4(d.s[j][i], sc[j][i]);
    }
    const int k0 = ch * kChunk;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + 64 * i;
      if (k >= K) break;  // uniform
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 xo;
        f32x4 sums = zero;
        prepare(k + 32 * h, x[i][h], xo, sums, sums);
#pragma unroll
        for (int j = 0; j < kSub; ++j) {
          const Operand w = operand(d.c, j, i, h);
          f32x4 D = O::mma(xo, w.b, k4 ? sums : zero);
          if (FMT == QW_FMT_NF4_B64) D = O::mma(xo, w.rest, D);
          scale_in(acc[j], FMT == QW_FMT_NF4_B64 || k4 ? sc[j][0][i] >> (k4 ? 16 * h : 0) : sc[j][h % CH::kScales][i], D, sums);
        }
      }
      load_x(min(k + kChunk, k_end - 64), x[i]);
    }
  }
  }
  if (FMT == QW_FMT_2BIT_G32) {
#pragma unroll
    for (int j = 0; j < kSub; ++j) acc[j] *= 0.01f;
  }

  if (ANCH) {
    // the anchor channels: 32 of them a step, the waves in turn from the
    // last, which has the fewest chunks. bf16 operands take the fp16 anchor
    // as two parts.
    for (int o0 = (kWaves - 1 - wv) * 32; o0 < a.n_out; o0 += kWaves * 32) {
      const int o = o0 + lg * 8;
      u32x4 A = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (o + q < a.n_out && (!few || ln < 4)) {  // few: in the rows of the first group
          int k = o + q;
          if (FMT == QW_FMT_2BIT_G32) {
            k = a.idx[(size_t)e * a.n_out + o + q];
            if ((uint32_t)k >= (uint32_t)K) k = 0;
          }
          A[q >> 1] |= (uint32_t)xp[k] << (16 * (q & 1));
        }
      }
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        u32x4 B = {0, 0, 0, 0}, B2 = {0, 0, 0, 0};
        if (wn[j] >= 0 && o < a.n_out_pad) {
          B = *reinterpret_cast<const u32x4 *>(a.wo + ((size_t)e * a.N + wn[j]) * a.n_out_pad + o);
          if (DT == QW_DT_BF16) split_f16(B, B2);
        }
        acc[j] = O::mma(A, B, acc[j]);
        if (DT == QW_DT_BF16) acc[j] = O::mma(A, B2, acc[j]);
      }
    }
  }

  // ---- the waves' sums, then one rounding ----
  __syncthreads();  // the table is done with
#pragma unroll
  for (int j = 0; j < kSub; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[wv][lg * 4 + r][j * 16 + ln] = acc[j][r];
  __syncthreads();
  const int row = tid >> 4;
  if (row >= rt.cnt) return;
  int yr = rt.p0 + row;
  if (a.by_slot) {
    yr = a.rows[yr];
    if ((uint32_t)yr >= (uint32_t)a.n) return;
  } else if (a.x_div && x_row(a.rows[yr], a.x_div, a.x_rows) < 0) {
    return;
  }
  auto total = [&](int c) {
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (few) {
#pragma unroll
        for (int g = 0; g < 4; ++g) v += *reinterpret_cast<const f32x4 *>(&part[w][4 * g + row][c]);
      } else {
        v += *reinterpret_cast<const f32x4 *>(&part[w][row][c]);
      }
    }
    return v;
  };
  const int c = (tid & 15) * 4;
  if (c >= half_cols) return;
  f32x4 v = total(c);
  if (a.swiglu) {
    const f32x4 u = total(c + kCols / 2);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = v[q] / (1.0f + expf(-v[q])) * u[q];
  }
  const int n = c0 + c;
  const size_t o = (size_t)yr * a.out_n + n;
  if (n + 4 <= a.out_n && a.out_n % 4 == 0) {
    if (a.y_dtype == QW_DT_F32)
      *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(a.Y) + o) = v;
    else
      *reinterpret_cast<u32x2 *>(reinterpret_cast<uint16_t *>(a.Y) + o) =
          u32x2{out_bits(v[0], a.y_dtype) | (out_bits(v[1], a.y_dtype) << 16),
                out_bits(v[2], a.y_dtype) | (out_bits(v[3], a.y_dtype) << 16)};
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (n + q >= a.out_n) continue;
      if (a.y_dtype == QW_DT_F32)
        reinterpret_cast<float *>(a.Y)[o + q] = v[q];
      else
        reinterpret_cast<uint16_t *>(a.Y)[o + q] = (uint16_t)out_bits(v[q], a.y_dtype);
    }
  }
}

// ---------------------------------------------------------------------------
// out[t][n] = sum_j weights[t][j] P[t * k + j][n] over the slots that are in
// a group: one read of the fp32 products, bound by memory. A thread takes
// four columns of one token.
struct CombineArgs {
  const float *P;  // [T * k][N]
  const int32_t *ids;
  const float *weights;
  void *out;
  int t0, k, N, E, dtype;  // t0: first token of the launch
  int col_blocks;
};

__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const int t = a.t0 + (int)(blockIdx.x / a.col_blocks);
  const int n = ((int)(blockIdx.x % a.col_blocks) * 256 + (int)threadIdx.x) * 4;
  if (n >= a.N) return;
  const bool vec = a.N % 4 == 0;
  f32x4 s = {0, 0, 0, 0};
  for (int j = 0; j < a.k; ++j) {
    const size_t slot = (size_t)t * a.k + j;
    if ((uint32_t)a.ids[slot] >= (uint32_t)a.E) continue;  // wave-uniform
    const float w = a.weights[slot];
    const float *p = a.P + slot * a.N + n;
    if (vec) {
      const f32x4 v = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] = __builtin_fmaf(w, v[q], s[q]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (n + q < a.N) s[q] = __builtin_fmaf(w, p[q], s[q]);
    }
  }
  const size_t o = (size_t)t * a.N + n;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (n + q >= a.N) continue;
    if (a.dtype == QW_DT_F32)
      reinterpret_cast<float *>(a.out)[o + q] = s[q];
    else
      reinterpret_cast<uint16_t *>(a.out)[o + q] = (uint16_t)out_bits(s[q], a.dtype);
  }
}

template <int FMT, int DT, bool ANCH>
qw_status launch_one(const ExpertArgs &a, hipStream_t s) {
  const long long grid = most_row_tiles(a.n, a.G, kRows) * a.col_tiles;
  if (grid > kMostBlocks) return QW_ERR_UNSUPPORTED;
  QW_HIP_TRY(launch(experts_kernel<FMT, DT, ANCH>, (unsigned)grid, kThreads, 0, s, a));
  return QW_OK;
}

template <int FMT, int DT>
qw_status launch_anch(const ExpertArgs &a, hipStream_t s) {
  if constexpr (FMT != QW_FMT_NF4_B64)
    if (a.n_out > 0) return launch_one<FMT, DT, true>(a, s);
  return launch_one<FMT, DT, false>(a, s);
}

template <int DT>
qw_status launch_fmt(int fmt, const ExpertArgs &a, hipStream_t s) {
  if (fmt == QW_FMT_2BIT_G32) return launch_anch<QW_FMT_2BIT_G32, DT>(a, s);
  if (fmt == QW_FMT_INT4_G32) return launch_anch<QW_FMT_INT4_G32, DT>(a, s);
  return launch_anch<QW_FMT_NF4_B64, DT>(a, s);
}

// 16-row blocks of a tile: the kernel whose estimated time is least.
//
// A kernel's time is a start plus a share per 256 workgroups (one a CU),
// the share (the narrow kernel's start too) growing with K; the tall tiles
// go by rounds, whole ones where they are few, each with its start. The rows per
// expert are on the device, so the number of row tiles is estimated: the
// rows by the tile's height and 0.6 of a short tile per expert, at least one
// for every expert that can have a row. The constants are fits, in us at K =
// 2048. Measured / estimated, bf16, experts x columns and the mean of their
// uneven rows (K = 2048; 8 experts: 4096), us:
//     2-bit                narrow   32 rows    64 rows   128 rows   256 rows
//     16 x 4096    16      37/37     50/47      50/59     41/34      59/60
//                  64      92/93     77/78      67/75     64/68      61/60
//                 128     158/166   115/119    100/103    69/68     120/120
//                 512               397/368    276/270   173/173    199/180
//      8 x 1024    32      21/24     61/65      81/87     57/64      86/116
//                 128      49/52     64/65      84/87     63/64      96/116
//     64 x 2816    32     135/140   119/115    124/115   100/102    163/180
//                 256               506/514    379/383   262/260    321/294
//      8 x 14336 1024              2223/2386  1601/1646  982/995    950/992
//     NF4
//     16 x 4096    16      44/40     45/42      44/53     57/43      72/73
//                  64     110/100    65/69      62/68     78/86      83/73
//                 128     204/180    99/104     92/94     82/86     156/146
//                 512               308/315    242/245   217/219    245/219
//      8 x 1024    32      27/25     63/58      69/78     98/82     127/142
//                 128      63/55     65/58      74/78    106/82     139/142
//     64 x 2816    32     171/151   103/100     96/104   141/129    226/219
//                 256               455/439    358/347   328/329    400/358
//      8 x 14336 1024              1992/2031  1464/1492 1253/1275  1165/1214
//     INT4
//     16 x 4096    16      44/43     45/41      60/53     44/40      62/66
//                  64     108/106    66/67      63/68     79/80     128/66
//                 128     199/189   103/103     94/94     79/80     133/132
//                 512               317/316    248/248   194/204    218/198
//      8 x 1024    32      26/30     60/57      70/78     69/76     100/128
//                 128      61/61     62/57      75/78     76/76     112/128
//     64 x 2816    32     166/159   106/99     120/105   118/120    190/198
//                 256               462/442    366/352   305/306    346/323
//      8 x 14336 1024              1986/2052  1554/1520 1211/1182  1055/1094
// It is off by a round where the rows need one tile more than a whole round
// (INT4, 16 x 4096, 64 rows: one expert had over 256).
struct Cost {
  float start, share;
};
int pick_row_blocks(int fmt, const ExpertArgs &a, bool tall) {
  constexpr int kHeights[5] = {1, 2, 4, 8, 16};
  constexpr Cost kCost[3][5] = {
      {{4, 4.6f}, {24, 20.7f}, {31, 27.8f}, {4, 30}, {4, 56}},  // 2-bit
      {{4, 5.0f}, {23, 17.6f}, {28, 25.2f}, {4, 39}, {4, 69}},  // NF4
      {{6, 5.2f}, {21, 17.8f}, {27, 25.7f}, {4, 36}, {4, 62}},  // INT4
  };
  const Cost *cost = kCost[fmt == QW_FMT_2BIT_G32 ? 0 : fmt == QW_FMT_NF4_B64 ? 1 : 2];
  double least = 1e30;
  int best = 1;
  for (int i = 0; i < (tall ? 5 : 3); ++i) {
    const int h = 16 * kHeights[i];
    const double tiles = fmax((double)a.n / h + 0.6 * a.G, fmin((double)a.n, (double)a.G));
    const double cols = ceil((double)a.N / (i == 0 ? kCols : 256));
    double rounds = fmax(fmin(tiles, (double)a.n) * cols / 256, i == 0 ? 0.0 : 1.0);
    if (i >= 3) rounds = rounds < 4 ? ceil(rounds) : rounds + 0.5;
    const double k = a.K / 2048.0, share = cost[i].share * rounds * k;
    const double t = i == 0 ? 4 + cost[i].start * k + share : cost[i].start * (i >= 3 ? rounds : 1.0) + share;
    if (t < least) {
      least = t;
      best = kHeights[i];
    }
  }
  return best;
}

// Argument checks the two entry points share; fills the weights' and rows'
// part of the arguments.
qw_status check_experts(const qw_experts *ew, const void *X, qw_dtype x_dtype, const qw_groups *g,
                        const void *Y, qw_dtype y_dtype, ExpertArgs *a) {
  if (!ew || !X || !Y || !g || ew->E < 1) return QW_ERR_INVALID_ARG;
  if (x_dtype != QW_DT_F16 && x_dtype != QW_DT_BF16) return QW_ERR_INVALID_ARG;
  if (!is_dtype(y_dtype)) return QW_ERR_INVALID_ARG;
  const qw_weight *w = &ew->w;
  if (w->format != QW_FMT_2BIT_G32 && w->format != QW_FMT_NF4_B64 && w->format != QW_FMT_INT4_G32)
    return QW_ERR_INVALID_ARG;
  QW_TRY(check_weight_view(w, w->format, 0));
  QW_TRY(check_groups(g));
  if (g->G != ew->E) return QW_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(Y)) return QW_ERR_ALIGNMENT;
  if (w->K % 64 || (unsigned long long)w->N * w->K >= (1ull << 32)) return QW_ERR_UNSUPPORTED;
  *a = ExpertArgs{};
  a->X = reinterpret_cast<const uint16_t *>(X);
  a->codes = w->codes;
  a->scales = reinterpret_cast<const uint8_t *>(w->scales);
  a->idx = w->out_idx;
  a->mask = w->out_mask;
  a->wo = w->out_w;
  a->offsets = g->offsets;
  a->rows = g->rows;
  a->G = g->G;
  a->n = g->n;
  a->N = a->out_n = w->N;
  a->K = w->K;
  a->n_out = w->format == QW_FMT_NF4_B64 ? 0 : w->n_out;
  a->n_out_pad = w->n_out_pad;
  const float *L = nf4_levels_host();
  for (int i = 0; i < 16; ++i) a->nf4[i] = L[i];
  return QW_OK;
}

qw_status run_experts(const qw_experts *ew, qw_dtype x_dtype, ExpertArgs &a, hipStream_t s) {
  const bool tall = experts_tall_fits(x_dtype, a);
  int blocks = tune(QW_TUNE_EXPERTS_ROW_BLOCKS);
  if (blocks < 1) blocks = pick_row_blocks(ew->w.format, a, tall);
  if (blocks > 4 && tall) return launch_experts_tall(ew->w.format, x_dtype, blocks, a, s);
  if (blocks > 1) return launch_experts_wide(ew->w.format, x_dtype, blocks, a, s);
  const int cols = a.swiglu ? kCols / 2 : kCols;
  a.col_tiles = (a.out_n + cols - 1) / cols;
  return x_dtype == QW_DT_F16 ? launch_fmt<QW_DT_F16>(ew->w.format, a, s)
                              : launch_fmt<QW_DT_BF16>(ew->w.format, a, s);
}

}  // namespace
}  // namespace qw

extern "C" {

qw_status qgemm_experts(const qw_experts *ew, const void *X, qw_dtype x_dtype, int x_rows, int x_div,
                        const qw_groups *g, int swiglu, void *Y, qw_dtype y_dtype, void *stream) {
  using namespace qw;
  CallScope scope;
  ExpertArgs a;
  QW_TRY(check_experts(ew, X, x_dtype, g, Y, y_dtype, &a));
  if (x_rows < 1 || x_div < 0 || (x_div == 0 && x_rows < g->n)) return QW_ERR_INVALID_ARG;
  if (swiglu && a.N % 2) return QW_ERR_INVALID_ARG;
  QW_TRY(current_device(nullptr));
  a.Y = Y;
  a.x_rows = x_rows;
  a.x_div = x_div;
  a.swiglu = swiglu != 0;
  if (a.swiglu) a.out_n = a.N / 2;
  a.y_dtype = y_dtype;
  return run_experts(ew, x_dtype, a, as_stream(stream));
}

size_t qw_experts_combine_workspace_bytes(int N, int T, int top_k) {
  if (N < 1 || T < 1 || top_k < 1 || (long long)T * top_k > QW_MAX_ROWS) return 0;
  return (size_t)T * (size_t)top_k * (size_t)N * sizeof(float);
}

qw_status qgemm_experts_combine(const qw_experts *ew, const void *H, qw_dtype h_dtype, const qw_groups *g,
                                const int32_t *ids, const float *weights, int T, int top_k, void *out,
                                qw_dtype out_dtype, void *workspace, size_t workspace_bytes, void *stream) {
  using namespace qw;
  CallScope scope;
  ExpertArgs a;
  QW_TRY(check_experts(ew, H, h_dtype, g, out, out_dtype, &a));
  if (!ids || !weights || T < 1 || top_k < 1 || (long long)T * top_k != g->n) return QW_ERR_INVALID_ARG;
  const size_t need = qw_experts_combine_workspace_bytes(a.N, T, top_k);
  if (!workspace || workspace_bytes < need) return QW_ERR_INVALID_ARG;
  if (!aligned16(ids) || !aligned16(weights) || !aligned16(workspace)) return QW_ERR_ALIGNMENT;
  QW_TRY(current_device(nullptr));
  const int col_blocks = (a.N + 1023) / 1024;
  a.Y = workspace;
  a.x_rows = g->n;
  a.x_div = 0;
  a.by_slot = 1;
  a.y_dtype = QW_DT_F32;
  QW_TRY(run_experts(ew, h_dtype, a, as_stream(stream)));
  // as many tokens a launch as its workgroups can be counted
  const int most = (int)(kMostBlocks / col_blocks);
  for (int t0 = 0; t0 < T; t0 += most) {
    const int now = T - t0 < most ? T - t0 : most;
    CombineArgs c{reinterpret_cast<const float *>(workspace), ids, weights, out, t0, top_k, a.N, ew->E, out_dtype, col_blocks};
    QW_HIP_TRY(launch(combine_kernel, (unsigned)(now * col_blocks), 256, 0, as_stream(stream), c));
  }
  return QW_OK;
}

}  // extern "C"
