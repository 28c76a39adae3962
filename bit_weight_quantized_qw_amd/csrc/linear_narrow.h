// The products of qgemm_linear by narrow tiles, for few rows. What bounds them: the packed weights' stream,
// read once; so the kernel is built to keep loads of codes in flight and to
// decode a weight in about one instruction. The scheme is the one of the
// experts' narrow tiles: a matrix instruction of 16 x 16 x 32 covers the 32
// weights of one scale group, the products are with the bare code levels and
// the group's scale multiplies the fp32 sum, so no weight is rounded (an NF4
// level is two 16-bit numbers).
//
// Tile: 16 MR rows times 64 columns, by four waves that each take a part of K;
// their sums meet in LDS in wave order.
#pragma once

#include "linear.h"

namespace qw {
namespace {

constexpr int kCols = 64;
constexpr int kSub = kCols / 16;  // 16-column blocks of a tile
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kChunk = 256;       // weights of one column in one set of loads

template <int FMT>
struct Chunk {
  static constexpr int kCodes = FMT == QW_FMT_2BIT_G32 ? 4 : 8;   // dwords
  static constexpr int kScales = FMT == QW_FMT_2BIT_G32 ? 2 : 1;  // dwords
  uint32_t c[kSub][kCodes];
  uint32_t s[kSub][kScales];
};

// Level table of the formats but INT4 (its entries as in the experts' narrow
// tiles: eight bytes a code byte, 16 replicas).
template <int FMT, int DT>
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

template <int FMT, int XT, bool ANCH, int MR>
__global__ __launch_bounds__(kThreads, 2) void narrow_kernel(LinearArgs a) {
  using XL = XLoad<XT>;
  constexpr int DT = XL::DT;
  using O = Op<DT>;
  constexpr bool k2 = FMT == QW_FMT_2BIT_G32, k4 = FMT == QW_FMT_INT4_G32, kN = FMT == QW_FMT_NF4_B64;
  constexpr int kSums = kWaves * 16 * (kCols + 4) * 4, kTable = k4 ? 0 : 256 * kEntry;
  __shared__ __attribute__((aligned(16))) char tab[kTable > kSums ? kTable : kSums];
  float(*const part)[16][kCols + 4] = reinterpret_cast<float(*)[16][kCols + 4]>(tab);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, lg = lane >> 4;
  const int ct = blockIdx.x % a.col_tiles, rt = blockIdx.x / a.col_tiles % a.row_tiles;
  const int part_of = blockIdx.x / (a.col_tiles * a.row_tiles);  // the part of K
  const int share = part_of * kWaves + wv, shares = a.parts * kWaves;
  const int m0 = rt * 16 * MR;
  const int K = a.K;

  // columns: gated tiles take 32 gate columns and the same 32 up columns
  const int half_cols = a.fin.gated ? kCols / 2 : kCols;
  const int c0 = ct * half_cols;
  constexpr int kCodeDiv = k2 ? 4 : 2;     // weights per code byte
  constexpr int kScaleDiv = k2 ? 8 : 16;   // weights per scale byte
  const auto rc = rsrc(a.codes, (uint32_t)((size_t)a.N * (K / kCodeDiv)));
  const auto rs = rsrc(a.scales, (uint32_t)((size_t)a.N * (K / kScaleDiv)));
  int wn[kSub];
#pragma unroll
  for (int j = 0; j < kSub; ++j) {
    const int h = c0 + (a.fin.gated ? (j & 1) : j) * 16 + ln;
    wn[j] = h < a.fin.out_n ? (a.fin.gated ? h + (j >> 1) * a.fin.out_n : h) : -1;
  }

  // this wave's chunks
  const int chunks = (K + kChunk - 1) / kChunk;
  const int ch0 = (int)((long long)chunks * share / shares), ch1 = (int)((long long)chunks * (share + 1) / shares);

  using CH = Chunk<FMT>;
  auto load = [&](int ch, CH &d) {
    const int k = ch * kChunk + lg * 64;
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      const bool in = k < K && wn[j] >= 0;
      const uint32_t oc = in ? (uint32_t)wn[j] * (uint32_t)(K / kCodeDiv) + (uint32_t)k / kCodeDiv : kOob;
      const uint32_t os = in ? (uint32_t)wn[j] * (uint32_t)(K / kScaleDiv) + (uint32_t)k / kScaleDiv : kOob;
#pragma unroll
      for (int i = 0; i < CH::kCodes; i += 4) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rc, (int)(in ? oc + 4 * i : kOob), 0, 0);
        d.c[j][i] = v[0]; d.c[j][i + 1] = v[1]; d.c[j][i + 2] = v[2]; d.c[j][i + 3] = v[3];
      }
      if (CH::kScales == 2) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rs, (int)os, 0, 0);
        d.s[j][0] = v[0];
        d.s[j][CH::kScales - 1] = v[1];
      } else {
        d.s[j][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)os, 0, 0);
      }
    }
  };

  // this lane's rows: those past M repeat the last one (and are not stored)
  size_t xrow[MR];
#pragma unroll
  for (int r = 0; r < MR; ++r) xrow[r] = (size_t)min(m0 + r * 16 + ln, a.M - 1) * K;

  f32x4 acc[MR][kSub];
#pragma unroll
  for (int r = 0; r < MR; ++r)
#pragma unroll
    for (int j = 0; j < kSub; ++j) acc[r][j] = f32x4{0, 0, 0, 0};
  const f32x4 zero = {0, 0, 0, 0};
  const uint32_t rep = (uint32_t)(lane & 15) * 8u;
  uint32_t sixteen = Int4<DT>::kSixteen;
  if (k4) asm volatile("" : "+v"(sixteen));  // an and-or takes one scalar operand
  auto entry = [&](uint32_t byte) { return tab + ((byte << 7) | rep); };

  struct Operand {
    u32x4 b, rest;  // NF4: the levels' second parts
  };
  auto operand = [&](const uint32_t (&c)[kSub][CH::kCodes], int j, int s, int h) {
    Operand o;
    if (k2) {
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

  CH next;
  if (ch0 < ch1) load(ch0, next);
  if (!k4) {
    fill_levels<FMT, DT>(tab, a.nf4);
    __syncthreads();
  }
#pragma unroll 1
  for (int ch = ch0; ch < ch1; ++ch) {
    CH d = next;
    if (ch + 1 < ch1) load(ch + 1, next);
    uint32_t sc[kSub][CH::kScales][4];
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      if (k2) to_halves(reinterpret_cast<uint32_t(&)[4]>(d.c[j][0]));
#pragma unroll
      for (int i = 0; i < CH::kCodes; i += 4) transpose4(reinterpret_cast<uint32_t(&)[4]>(d.c[j][i]));
#pragma unroll
      for (int i = 0; i < CH::kScales; ++i) gather4(d.s[j][i], sc[j][i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (ch * kChunk + 64 * i >= K) break;  // uniform
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = ch * kChunk + 64 * i + 32 * h;
        u32x4 x[MR];
        f32x4 sums[MR];
#pragma unroll
        for (int r = 0; r < MR; ++r) {
          x[r] = XL::operand(XL::load(a.X, xrow[r] + k + lg * 8));
          sums[r] = zero;
          if (k2) {  // 100 times the row sums of x, for Z
            if (ANCH) {
              const uint32_t m = a.mask[k / 32] >> (8 * lg);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                x[r][q] &= ~(((m >> (2 * q)) & 1 ? 0xFFFFu : 0u) | ((m >> (2 * q + 1)) & 1 ? 0xFFFF0000u : 0u));
            }
            const uint32_t hundred = O::bits(100.0f) * 0x10001u;
            sums[r] = O::mma(x[r], u32x4{hundred, hundred, hundred, hundred}, zero);
          }
          if (k4) {  // -24 times them, so that 16 + u counts as u - 8
            x[r] = Int4<DT>::order(x[r]);
            constexpr uint32_t m24 = Int4<DT>::kMinus24;
            sums[r] = O::mma(x[r], u32x4{m24, m24, m24, m24}, zero);
          }
        }
#pragma unroll
        for (int j = 0; j < kSub; ++j) {
          const Operand w = operand(d.c, j, i, h);
          const uint32_t sw = kN || k4 ? sc[j][0][i] >> (k4 ? 16 * h : 0) : sc[j][h % CH::kScales][i];
          const float S = kN ? __builtin_bit_cast(float, sw) : f16_bits_to_f32((uint16_t)sw);
          const float Z = f16_bits_to_f32((uint16_t)(sw >> 16));
#pragma unroll
          for (int r = 0; r < MR; ++r) {
            f32x4 D = O::mma(x[r], w.b, k4 ? sums[r] : zero);
            if (kN) D = O::mma(x[r], w.rest, D);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              acc[r][j][q] = __builtin_fmaf(S, D[q], k2 ? __builtin_fmaf(Z, sums[r][q], acc[r][j][q]) : acc[r][j][q]);
          }
        }
      }
    }
  }
  if (k2) {
#pragma unroll
    for (int r = 0; r < MR; ++r)
#pragma unroll
      for (int j = 0; j < kSub; ++j) acc[r][j] *= 0.01f;
  }

  if (ANCH) {
    // the anchor channels: 32 of them a step, the waves in turn. bf16
    // operands take the fp16 anchor as two parts.
    for (int o0 = share * 32; o0 < a.n_out; o0 += shares * 32) {
      const int o = o0 + lg * 8;
      u32x4 A[MR];
#pragma unroll
      for (int r = 0; r < MR; ++r) A[r] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (o + q < a.n_out) {
          int k = o + q;
          if (k2) {
            k = a.idx[o + q];
            if ((uint32_t)k >= (uint32_t)K) k = 0;
          }
#pragma unroll
          for (int r = 0; r < MR; ++r) A[r][q >> 1] |= one_as_16<XT, DT>(a.X, xrow[r] + k) << (16 * (q & 1));
        }
      }
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        u32x4 B = {0, 0, 0, 0}, B2 = {0, 0, 0, 0};
        if (wn[j] >= 0 && o < a.n_out_pad) {
          B = *reinterpret_cast<const u32x4 *>(a.wo + (size_t)wn[j] * a.n_out_pad + o);
          if (DT == QW_DT_BF16) split_f16(B, B2);
        }
#pragma unroll
        for (int r = 0; r < MR; ++r) {
          acc[r][j] = O::mma(A[r], B, acc[r][j]);
          if (DT == QW_DT_BF16) acc[r][j] = O::mma(A[r], B2, acc[r][j]);
        }
      }
    }
  }

  // ---- the waves' sums of one block of 16 rows at a time, then what follows ----
  const int row = tid >> 4, c = (tid & 15) * 4;
#pragma unroll
  for (int r = 0; r < MR; ++r) {
    __syncthreads();  // the table, or the block before, is done with
#pragma unroll
    for (int j = 0; j < kSub; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) part[wv][lg * 4 + q][j * 16 + ln] = acc[r][j][q];
    __syncthreads();
    const int m = m0 + r * 16 + row;
    if (m >= a.M || c >= half_cols || c0 + c >= a.fin.out_n) continue;
    auto total = [&](int at) {
      f32x4 v = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += *reinterpret_cast<const f32x4 *>(&part[w][row][at]);
      return v;
    };
    f32x4 up = zero;
    if (a.fin.gated) up = total(c + kCols / 2);
    if (a.parts > 1) {
      store_part(a.fin, part_of, m, c0 + c, a.fin.out_n, total(c));
      if (a.fin.gated) store_part(a.fin, part_of, m, a.fin.out_n + c0 + c, a.N, up);
    } else {
      const f32x4 v = shape_values(a.fin, total(c), up, scale_at(a.fin, m), bias_at(a.fin, c0 + c), bias_up_at(a.fin, c0 + c));
      store_four(a.fin, m, c0 + c, v + residual_at(a.fin, m, c0 + c));
    }
  }
}

template <int FMT, int XT, bool ANCH, int MR>
qw_status launch_one(LinearArgs a, hipStream_t s) {
  const int cols = a.fin.gated ? kCols / 2 : kCols;
  a.col_tiles = (a.fin.out_n + cols - 1) / cols;
  a.row_tiles = (a.M + 16 * MR - 1) / (16 * MR);
  const long long grid = (long long)a.col_tiles * a.row_tiles * a.parts;
  if (grid > kMostBlocks) return QW_ERR_UNSUPPORTED;
  QW_HIP_TRY(launch(narrow_kernel<FMT, XT, ANCH, MR>, (unsigned)grid, kThreads, 0, s, a));
  return QW_OK;
}

template <int FMT, int XT, bool ANCH>
qw_status launch_rows(const LinearArgs &a, int row_blocks, hipStream_t s) {
  return row_blocks == 1 ? launch_one<FMT, XT, ANCH, 1>(a, s) : launch_one<FMT, XT, ANCH, 2>(a, s);
}

template <int FMT, int XT>
qw_status launch_anch(const LinearArgs &a, int row_blocks, hipStream_t s) {
  if constexpr (FMT != QW_FMT_NF4_B64)
    if (a.n_out > 0) return launch_rows<FMT, XT, true>(a, row_blocks, s);
  return launch_rows<FMT, XT, false>(a, row_blocks, s);
}

}  // namespace

template <int FMT>
qw_status launch_linear_narrow(const LinearArgs &a, int row_blocks, hipStream_t s) {
  switch (a.x_dtype) {
    case QW_DT_F16: return launch_anch<FMT, QW_DT_F16>(a, row_blocks, s);
    case QW_DT_BF16: return launch_anch<FMT, QW_DT_BF16>(a, row_blocks, s);
    case QW_DT_E4M3: return launch_anch<FMT, QW_DT_E4M3>(a, row_blocks, s);
    default: return launch_anch<FMT, QW_DT_I8>(a, row_blocks, s);
  }
}

}  // namespace qw
