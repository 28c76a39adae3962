// The products of qgemm_linear by narrow tiles, for few rows. What should bound
// them is the packed weights' stream, read once; so the kernel is built to keep
// loads of codes in flight and to decode a weight in about one instruction. The scheme is the one of the
// experts' narrow tiles: a matrix instruction of 16 x 16 x 32 covers the 32
// weights of one scale group, the products are with the bare code levels and
// the group's scale multiplies the fp32 sum, so no weight is rounded (an NF4
// level is two 16-bit numbers).
//
// Tile: 4 or 16 MR rows times 16 SUB columns, by W waves that each take a part
// of K; their sums meet in LDS in wave order.
//
// Measured, 7 rows of 8192 x 28672: INT4 with anchors and e4m3 rows 42 us (3.2
// TB/s), NF4 41, 2-bit with anchors 59; one row in NF4 33. What bounds them: the
// loads' address units, busy 0.58 of the cycles in the first of these, beside 0.38
// of vector issue and 0.09 of matrix products. A load touches 16 rows because a lane
// takes the column whose operand it holds; consecutive bytes of one row by a run of
// lanes, turned in LDS, would touch fewer, and have not been tried here.
#pragma once

#include "linear.h"

namespace qw {
namespace {

constexpr int kChunk = 256;       // weights of one column in one set of loads

template <int FMT, int SUB>
struct Chunk {
  static constexpr int kCodes = FMT == QW_FMT_2BIT_G32 ? 4 : 8;   // dwords
  static constexpr int kScales = FMT == QW_FMT_2BIT_G32 ? 2 : 1;  // dwords
  uint32_t c[SUB][kCodes];
  uint32_t s[SUB][kScales];
};

// Level table of the formats but INT4 (its entries as in the experts' narrow
// tiles: eight bytes a code byte, 16 replicas).
template <int FMT, int DT, int kThreads>
__device__ inline void fill_levels(char *tab, const float *nf4) {
  for (int v = threadIdx.x; v < 256; v += kThreads) {
    u32x2 w;
    if (FMT == QW_FMT_2BIT_G32) {
      uint32_t l[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int q = (v >> (2 * t)) & 3;
        l[t] = Op<DT>::bits(q == 0 ? -152.0f : q == 1 ? -45.0f : q == 2 ? 45.0f : 152.0f);
      }
      w = u32x2{l[0] | (l[1] << 16), l[2] | (l[3] << 16)};
    } else {
      const float lo = nf4[v & 15], hi = nf4[v >> 4];
      const uint32_t lo16 = Op<DT>::bits(lo), hi16 = Op<DT>::bits(hi);
      w = u32x2{lo16 | (hi16 << 16),
                Op<DT>::bits(lo - Op<DT>::value(lo16)) | (Op<DT>::bits(hi - Op<DT>::value(hi16)) << 16)};
    }
#pragma unroll
    for (int r = 0; r < 8; ++r)
      *reinterpret_cast<u32x4 *>(tab + v * kEntry + ((r + v) & 7) * 16) = u32x4{w[0], w[1], w[0], w[1]};
  }
}

// 16 MR rows times 16 SUB columns by W waves; MR = 0: up to four rows.
//
// Up to four rows: operand row 4 s + m is row m of X in the s-th of four
// consecutive scale groups and zero in the others, so four products run into
// one result, whose rows lane group s holds for its own group: one scaling per
// four products, by a scale word that only that lane group needs, and a
// quarter of the loads of X. The groups' sums are added up with the waves'.
template <int FMT, int XT, bool ANCH, int MR, int SUB, int W>
__global__ __launch_bounds__(64 * W) void narrow_kernel(LinearArgs a) {
  using XL = XLoad<XT>;
  constexpr int DT = XL::DT;
  using O = Op<DT>;
  constexpr bool k2 = FMT == QW_FMT_2BIT_G32, k4 = FMT == QW_FMT_INT4_G32, kN = FMT == QW_FMT_NF4_B64;
  constexpr int kCols = 16 * SUB, kThreads = 64 * W;
  constexpr bool kFew = MR == 0;
  constexpr int R = kFew ? 1 : MR;        // 16-row blocks of operands
  constexpr int kHigh = kFew ? 4 : 16 * MR;
  constexpr int kRuns = 4;  // runs of 64 elements of X that are on their way
  static_assert(!kFew || !k4, "INT4 takes tiles of 16 rows");
  constexpr int kSums = W * 16 * (kCols + 4) * 4, kTable = k4 ? 0 : 256 * kEntry;
  __shared__ __attribute__((aligned(16))) char tab[kTable > kSums ? kTable : kSums];
  float(*const part)[16][kCols + 4] = reinterpret_cast<float(*)[16][kCols + 4]>(tab);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, lg = lane >> 4;
  const int ct = blockIdx.x % a.col_tiles, rt = blockIdx.x / a.col_tiles % a.row_tiles;
  const int part_of = blockIdx.x / (a.col_tiles * a.row_tiles);  // the part of K
  const int share = part_of * W + wv, shares = a.parts * W;
  const int m0 = rt * kHigh;
  const int K = a.K;

  // columns: gated tiles take the same columns of gate and up
  const int half_cols = a.fin.gated ? kCols / 2 : kCols;
  const int c0 = ct * half_cols;
  constexpr int kCodeDiv = k2 ? 4 : 2;     // weights per code byte
  constexpr int kScaleDiv = k2 ? 8 : 16;   // weights per scale byte
  const auto rc = rsrc(a.codes, (uint32_t)((size_t)a.N * (K / kCodeDiv)));
  const auto rs = rsrc(a.scales, (uint32_t)((size_t)a.N * (K / kScaleDiv)));
  int wn[SUB];
#pragma unroll
  for (int j = 0; j < SUB; ++j) {
    constexpr int kHalf = SUB > 1 ? SUB / 2 : 1;
    const int h = c0 + (a.fin.gated ? j % kHalf : j) * 16 + ln;
    wn[j] = h < a.fin.out_n ? (a.fin.gated ? h + j / kHalf * a.fin.out_n : h) : -1;
  }

  // this wave's chunks
  const int chunks = (K + kChunk - 1) / kChunk;
  const int ch0 = (int)((long long)chunks * share / shares), ch1 = (int)((long long)chunks * (share + 1) / shares);

  using CH = Chunk<FMT, SUB>;
  auto load = [&](int ch, CH &d) {
    const int k = ch * kChunk + lg * 64;
#pragma unroll
    for (int j = 0; j < SUB; ++j) {
      const bool in = k < K && wn[j] >= 0;
      const uint32_t os = in ? (uint32_t)wn[j] * (uint32_t)(K / kScaleDiv) + (uint32_t)k / kScaleDiv : kOob;
#pragma unroll
      for (int i = 0; i < CH::kCodes; i += 4) {
        // the four lane groups' pieces of a column side by side: of 2-bit codes 64
        // weights each, of 4-bit ones the group lg (then 4 + lg) of 32
        const int kc = k2 ? k : ch * kChunk + i * 32 + lg * 32;
        const uint32_t oc = (uint32_t)max(wn[j], 0) * (uint32_t)(K / kCodeDiv) + (uint32_t)kc / kCodeDiv;
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rc, (int)(wn[j] >= 0 && kc < K ? oc : kOob), 0, 0);
        d.c[j][i] = v[0]; d.c[j][i + 1] = v[1]; d.c[j][i + 2] = v[2]; d.c[j][i + 3] = v[3];
      }
      if (kFew && !kN) continue;  // load_few_scales
      if (CH::kScales == 2) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rs, (int)os, 0, 0);
        d.s[j][0] = v[0];
        d.s[j][CH::kScales - 1] = v[1];
      } else {
        d.s[j][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)os, 0, 0);
      }
    }
  };

  // this lane's rows; those past M are not asked for and read as zeros (a load's
  // time goes by the lines that its lanes ask for: one row by 8192 x 28672 in NF4
  // 36.0 us with the last row repeated in their place, 33.8 so)
  const int rows = min(kHigh, a.M - m0);
  const auto rx = rsrc(reinterpret_cast<const char *>(a.X) + (size_t)m0 * K * XL::kBytes, (uint32_t)rows * (uint32_t)K * XL::kBytes);
  uint32_t xo[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = r * 16 + (kFew ? ln & 3 : ln);
    xo[r] = row < rows ? ((uint32_t)row * (uint32_t)K + lg * 8) * XL::kBytes : kOob;
  }
  // with 64 elements of X come the anchor bits of their channels (through the
  // vector memory path: a scalar load would be waited for at every use)
  const auto rm = rsrc(a.mask, ANCH && k2 ? (uint32_t)K / 8 : 0);
  struct XRun {
    typename XL::raw v[2][R];
    uint32_t drop[2];
  };
  // run of 64 elements from k on, or where there is none the last one (unused)
  auto load_x = [&](int k, XRun &d) {
    const int at = min(k, K - 64);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < R; ++r) d.v[h][r] = XL::load(rx, xo[r], (at + 32 * h) * XL::kBytes);
    if (k2 && ANCH) {
      int o = at / 8;
      asm volatile("" : "+v"(o));
      const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(rm, o, 0, 0);
      d.drop[0] = w[0];
      d.drop[1] = w[1];
    }
  };
  // up to four rows: the two pieces of a chunk's elements that this lane's
  // operand row holds, those of groups slot and slot + 4 (NF4: of its block)
  const int slot = ln >> 2;
  auto load_few = [&](int ch, XRun &d) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = kN ? ch * kChunk + slot * 64 + q * 32 : ch * kChunk + (q * 4 + slot) * 32;
      d.v[q][0] = XL::load(rx, k < K ? xo[0] + k * XL::kBytes : kOob, 0);  // past K: 0
      if (k2 && ANCH) d.drop[q] = __builtin_amdgcn_raw_buffer_load_b32(rm, k / 8, 0, 0);  // past K: 0
    }
  };
  auto without_anchors = [&](u32x4 v, uint32_t word) {
    const uint32_t m = word >> (8 * lg);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] &= ~(((m >> (2 * q)) & 1 ? 0xFFFFu : 0u) | ((m >> (2 * q + 1)) & 1 ? 0xFFFF0000u : 0u));
    return v;
  };

  f32x4 acc[R][SUB];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < SUB; ++j) acc[r][j] = f32x4{0, 0, 0, 0};
  const f32x4 zero = {0, 0, 0, 0};
  const uint32_t rep = (uint32_t)(lane & 15) * 8u;
  uint32_t sixteen = Int4<DT>::kSixteen;
  if (k4) asm volatile("" : "+v"(sixteen));  // an and-or takes one scalar operand
  auto entry = [&](uint32_t byte) { return tab + ((byte << 7) | rep); };

  struct Operand {
    u32x4 b, rest;  // NF4: the levels' second parts
  };
  auto operand = [&](const uint32_t (&c)[SUB][CH::kCodes], int j, int s, int h) {
    Operand o;
    if (k2) {
      const uint32_t w = c[j][s] >> (16 * h);
      const u32x2 lo = *reinterpret_cast<const u32x2 *>(entry(w & 0xFFu));
      const u32x2 hi = *reinterpret_cast<const u32x2 *>(entry((w >> 8) & 0xFFu));
      o.b = u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else if (k4) {
      o.b = Int4<DT>::operand(c[j][(2 * s + h) % CH::kCodes], sixteen);
    } else {
      const uint32_t w = c[j][(2 * s + h) % CH::kCodes];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const u32x2 l = *reinterpret_cast<const u32x2 *>(entry((w >> (8 * q)) & 0xFFu));
        o.b[q] = l[0];
        o.rest[q] = l[1];
      }
    }
    return o;
  };

  // 2-bit scale words of a few rows: those of groups lg and 4 + lg of the chunk
  auto load_few_scales = [&](int ch, CH &d) {
    if (!kFew || !k2) return;
    const int g = ch * (kChunk / 32) + lg;
#pragma unroll
    for (int j = 0; j < SUB; ++j) {
      const uint32_t at = (uint32_t)max(wn[j], 0) * (uint32_t)(K / kScaleDiv) + (uint32_t)g * 4;
      const uint32_t o0 = wn[j] >= 0 && g < K / 32 ? at : kOob, o1 = wn[j] >= 0 && g + 4 < K / 32 ? at + 16 : kOob;
      d.s[j][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)o0, 0, 0);
      d.s[j][CH::kScales - 1] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)o1, 0, 0);
    }
  };
  CH next;
  XRun x[kFew ? 1 : kRuns];
  if (ch0 < ch1) {
    load(ch0, next);
    load_few_scales(ch0, next);
    if constexpr (kFew) {
      load_few(ch0, x[0]);
    } else {
#pragma unroll
      for (int i = 0; i < kRuns; ++i) load_x(ch0 * kChunk + 64 * i, x[i]);
    }
  }
  // what stands behind the sums: this thread's row and columns of them
  const int row = tid / (4 * SUB), c = tid % (4 * SUB) * 4;
  const bool mine = row < (kFew ? 4 : 16) && c < half_cols && c0 + c < a.fin.out_n;
  f32x4 bias = zero, bias_up = zero, residual = zero;
  float scale = 1.0f;
  auto ask = [&](int m) {
    scale = scale_at(a.fin, m);
    residual = residual_at(a.fin, m, c0 + c);
  };
  if (a.parts == 1 && mine) {
    bias = bias_at(a.fin, c0 + c);
    bias_up = bias_up_at(a.fin, c0 + c);
    if (m0 + row < a.M) ask(m0 + row);
  }
  if (!k4) {
    fill_levels<FMT, DT, kThreads>(tab, a.nf4);
    __syncthreads();
  }
  if (ANCH) {
    // the anchor channels, while the first codes are on their way: 32 of them a
    // step, the waves in turn. bf16 operands take the fp16 anchor as two parts.
    const auto ri = rsrc(a.idx, k2 ? (uint32_t)a.n_out * 4u : 0u);
    for (int o0 = share * 32; o0 < a.n_out; o0 += shares * 32) {
      const int o = o0 + lg * 8;
      u32x4 at[2];
      if (k2) {  // past the last: channel 0
        at[0] = __builtin_amdgcn_raw_buffer_load_b128(ri, o * 4, 0, 0);
        at[1] = __builtin_amdgcn_raw_buffer_load_b128(ri, o * 4 + 16, 0, 0);
      }
      u32x4 B[SUB], B2[SUB];
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
        B[j] = B2[j] = u32x4{0, 0, 0, 0};
        if (wn[j] >= 0 && o < a.n_out_pad) B[j] = *reinterpret_cast<const u32x4 *>(a.wo + (size_t)wn[j] * a.n_out_pad + o);
      }
      u32x4 A[R];
#pragma unroll
      for (int r = 0; r < R; ++r) A[r] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        uint32_t k = (uint32_t)(o + q);
        if (k2) k = at[q >> 2][q & 3] < (uint32_t)K ? at[q >> 2][q & 3] : 0u;
        const bool in = o + q < a.n_out && (!kFew || ln < 4);  // few: in the rows of the first group
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (in && xo[r] != kOob)
            A[r][q >> 1] |= one_as_16<XT, DT>(a.X, (size_t)(m0 + r * 16 + (kFew ? ln & 3 : ln)) * K + k) << (16 * (q & 1));
      }
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
        if (DT == QW_DT_BF16) split_f16(B[j], B2[j]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          acc[r][j] = O::mma(A[r], B[j], acc[r][j]);
          if (DT == QW_DT_BF16) acc[r][j] = O::mma(A[r], B2[j], acc[r][j]);
        }
      }
    }
    if (k2) {  // levels are a hundredfold
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < SUB; ++j) acc[r][j] *= 100.0f;
    }
  }
  if constexpr (kFew) {
    constexpr int kGroup = kN ? 64 : 32, kQuads = kChunk / (4 * kGroup);
#pragma unroll 1
    for (int ch = ch0; ch < ch1; ++ch) {
      CH d = next;
      XRun xr = x[0];
      if (ch + 1 < ch1) {
        load(ch + 1, next);
        load_few_scales(ch + 1, next);
        load_few(ch + 1, x[0]);
      }
      u32x4 xo[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        xo[q] = XL::operand(xr.v[q][0]);
        if (k2 && ANCH) xo[q] = without_anchors(xo[q], xr.drop[q]);
      }
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
        if (k2) to_halves(reinterpret_cast<uint32_t(&)[4]>(d.c[j][0]));
#pragma unroll
        for (int i = 0; i < CH::kCodes; i += 4) transpose4(reinterpret_cast<uint32_t(&)[4]>(d.c[j][i]));
      }
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        f32x4 sums = zero, D[SUB];
#pragma unroll
        for (int j = 0; j < SUB; ++j) D[j] = zero;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
          for (int h = 0; h < (kN ? 2 : 1); ++h) {
            u32x4 A = xo[kN ? h : q];
#pragma unroll
            for (int t = 0; t < 4; ++t) A[t] = slot == s ? A[t] : 0u;
            const uint32_t hundred = O::bits(100.0f) * 0x10001u;
            if (k2) sums = O::mma(A, u32x4{hundred, hundred, hundred, hundred}, sums);
            // step (32 weights) 4 q + s of the chunk; NF4: 2 s + h
            const int step = kN ? 2 * s + h : 4 * q + s;
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
              const Operand w = operand(d.c, j, step >> 1, step & 1);
              D[j] = O::mma(A, w.b, D[j]);
              if (kN) D[j] = O::mma(A, w.rest, D[j]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
          const uint32_t sw = d.s[j][q % CH::kScales];
          const float S = kN ? __builtin_bit_cast(float, sw) : f16_bits_to_f32((uint16_t)sw);
          const float Z = f16_bits_to_f32((uint16_t)(sw >> 16));
#pragma unroll
          for (int t = 0; t < 4; ++t)
            acc[0][j][t] = __builtin_fmaf(S, D[j][t], k2 ? __builtin_fmaf(Z, sums[t], acc[0][j][t]) : acc[0][j][t]);
        }
      }
    }
  } else {
#pragma unroll 1
  for (int ch = ch0; ch < ch1; ++ch) {
    CH d = next;
    if (ch + 1 < ch1) load(ch + 1, next);
    uint32_t sc[SUB][CH::kScales][4];
#pragma unroll
    for (int j = 0; j < SUB; ++j) {
      if (k2) to_halves(reinterpret_cast<uint32_t(&)[4]>(d.c[j][0]));
#pragma unroll
      for (int i = 0; i < CH::kCodes; i += 4) transpose4(reinterpret_cast<uint32_t(&)[4]>(d.c[j][i]));
#pragma unroll
      for (int i = 0; i < CH::kScales; ++i) gather4(d.s[j][i], sc[j][i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k0 = ch * kChunk + 64 * i;
      if (k0 >= K) break;  // uniform
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 xo[R];
        f32x4 sums[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          xo[r] = XL::operand(x[i % kRuns].v[h][r]);
          sums[r] = zero;
          if (k2) {  // 100 times the row sums of x, for Z
            if (ANCH) xo[r] = without_anchors(xo[r], x[i % kRuns].drop[h]);
            const uint32_t hundred = O::bits(100.0f) * 0x10001u;
            sums[r] = O::mma(xo[r], u32x4{hundred, hundred, hundred, hundred}, zero);
          }
          if (k4) {  // -24 times them, so that 16 + u counts as u - 8
            xo[r] = Int4<DT>::order(xo[r]);
            constexpr uint32_t m24 = Int4<DT>::kMinus24;
            sums[r] = O::mma(xo[r], u32x4{m24, m24, m24, m24}, zero);
          }
        }
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
          const Operand w = operand(d.c, j, i, h);
          const uint32_t sw = kN || k4 ? sc[j][0][i] >> (k4 ? 16 * h : 0) : sc[j][h % CH::kScales][i];
          const float S = kN ? __builtin_bit_cast(float, sw) : f16_bits_to_f32((uint16_t)sw);
          const float Z = f16_bits_to_f32((uint16_t)(sw >> 16));
#pragma unroll
          for (int r = 0; r < R; ++r) {
            f32x4 D = O::mma(xo[r], w.b, k4 ? sums[r] : zero);
            if (kN) D = O::mma(xo[r], w.rest, D);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              acc[r][j][q] = __builtin_fmaf(S, D[q], k2 ? __builtin_fmaf(Z, sums[r][q], acc[r][j][q]) : acc[r][j][q]);
          }
        }
      }
      load_x(k0 + 64 * kRuns, x[i % kRuns]);  // past this wave's share: unused
    }
  }
  }
  if (k2) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < SUB; ++j) acc[r][j] *= 0.01f;
  }

  // ---- the waves' sums of one block of 16 rows at a time, then what follows ----
#pragma unroll
  for (int r = 0; r < R; ++r) {
    __syncthreads();  // the table, or the block before, is done with
#pragma unroll
    for (int j = 0; j < SUB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) part[wv][lg * 4 + q][j * 16 + ln] = acc[r][j][q];
    __syncthreads();
    const int m = m0 + r * 16 + row;
    if (m >= a.M || !mine) continue;
    auto total = [&](int at) {
      f32x4 v = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if constexpr (kFew) {
#pragma unroll
          for (int g = 0; g < 4; ++g) v += *reinterpret_cast<const f32x4 *>(&part[w][4 * g + row][at]);
        } else {
          v += *reinterpret_cast<const f32x4 *>(&part[w][row][at]);
        }
      }
      return v;
    };
    f32x4 up = zero;
    if (a.fin.gated) up = total(c + kCols / 2);
    if (a.parts > 1) {
      store_part(a.fin, part_of, m, c0 + c, a.fin.out_n, total(c));
      if (a.fin.gated) store_part(a.fin, part_of, m, a.fin.out_n + c0 + c, a.N, up);
    } else {
      const f32x4 v = shape_values(a.fin, total(c), up, scale, bias, bias_up) + residual;
      if (r + 1 < R && m + 16 < a.M) ask(m + 16);
      store_four(a.fin, m, c0 + c, v);
    }
  }
}

template <int FMT, int XT, bool ANCH, int MR, int SUB, int W>
qw_status launch_one(LinearArgs a, hipStream_t s) {
  if (SUB == 1 && a.fin.gated) return QW_ERR_UNSUPPORTED;  // such a tile has no up columns
  const int cols = a.fin.gated ? 8 * SUB : 16 * SUB;
  a.col_tiles = (a.fin.out_n + cols - 1) / cols;
  constexpr int kHigh = MR == 0 ? 4 : 16 * MR;
  a.row_tiles = (a.M + kHigh - 1) / kHigh;
  const long long grid = (long long)a.col_tiles * a.row_tiles * a.parts;
  if (grid * W > kMostBlocks * 4) return QW_ERR_UNSUPPORTED;
  QW_HIP_TRY(launch(narrow_kernel<FMT, XT, ANCH, MR, SUB, W>, (unsigned)grid, 64 * W, 0, s, a));
  return QW_OK;
}

// shape: rows (0: up to four, else 16-row blocks), columns / 16 and waves, as
// decimal digits (the choice is pick_narrow's, linear.hip).
template <int FMT, int XT, bool ANCH>
qw_status launch_shape(const LinearArgs &a, int shape, hipStream_t s) {
#define QW_SHAPE(MR, SUB, W) \
  if (shape == narrow_shape(MR, SUB, W)) return launch_one<FMT, XT, ANCH, MR, SUB, W>(a, s);
  if constexpr (FMT != QW_FMT_INT4_G32) {
    QW_SHAPE(0, 1, 8)
    QW_SHAPE(0, 2, 4)
    QW_SHAPE(0, 2, 8)
    QW_SHAPE(0, 2, 16)
  }
  QW_SHAPE(1, 2, 8)
  QW_SHAPE(1, 4, 4)
  QW_SHAPE(1, 4, 8)
  QW_SHAPE(2, 2, 8)
  QW_SHAPE(2, 4, 8)
#undef QW_SHAPE
  return QW_ERR_UNSUPPORTED;
}

template <int FMT, int XT>
qw_status launch_anch(const LinearArgs &a, int shape, hipStream_t s) {
  if constexpr (FMT != QW_FMT_NF4_B64)
    if (a.n_out > 0) return launch_shape<FMT, XT, true>(a, shape, s);
  return launch_shape<FMT, XT, false>(a, shape, s);
}

}  // namespace

template <int FMT>
qw_status launch_linear_narrow(const LinearArgs &a, int shape, hipStream_t s) {
  switch (a.x_dtype) {
    case QW_DT_F16: return launch_anch<FMT, QW_DT_F16>(a, shape, s);
    case QW_DT_BF16: return launch_anch<FMT, QW_DT_BF16>(a, shape, s);
    case QW_DT_E4M3: return launch_anch<FMT, QW_DT_E4M3>(a, shape, s);
    default: return launch_anch<FMT, QW_DT_I8>(a, shape, s);
  }
}

}  // namespace qw
