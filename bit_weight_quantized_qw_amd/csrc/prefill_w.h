// The prefill GEMM that keeps W out of LDS, for one matrix (prefill.hip) and
// for rows grouped by expert (experts_tall.hip).
#pragma once

#include <type_traits>

#include "op16.h"
#include "row_groups.h"

namespace qw {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));

constexpr int BM = 256, BN = 256, BK = 64;
constexpr int LDA = BK + 8;  // bf16 elements per LDS row (144 bytes)
constexpr int NT = 256;

struct PrefillArgs {
  static constexpr bool kGrouped = false;
  static constexpr int kRows = BM;  // rows of a tile
  static constexpr int kType = QW_DT_BF16;  // of X, of the weights as they enter, of 16-bit Y
  const uint16_t *X;       // [M][K] bf16
  const uint32_t *codes;   // 2-bit: [N][K/16]; NF4, INT4: [N][K/8]
  const void *scales;      // 2-bit: uint32 [N][K/32]; NF4: float [N][K/64]; INT4: fp16 [N][K/32]
  const int32_t *idx;      // anchors (2-bit), may be null
  const uint16_t *wo;      // [N][n_out_pad]
  void *Y;                 // [M][N]
  int M, N, K, n_out, n_out_pad;
  int mt_count;            // number of 256-row tiles along M
  int n_begin;             // first output column of this launch's tiles
  int xcd_group;           // row tiles per group of the XCD-aware tile order (0: plain order)
  float nf4[16];           // level of each 4-bit code (NF4 table; u - 8 for INT4)
};

// The same product for rows grouped by expert, tiles of ROWS rows: codes and
// scales are those of expert 0, M is the number of rows of X, and Y has a row
// for each of the n positions.
template <int ROWS, int DT>
struct GroupedArgs : PrefillArgs {
  static constexpr bool kGrouped = true;
  static constexpr int kRows = ROWS;
  static constexpr int kType = DT;
  const int32_t *offsets, *rows;
  int G, n, x_div, by_slot;
  int n_tiles;             // column tiles of this launch
};

__device__ inline uint32_t f32_to_bf16_bits(float v) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// RNE of both values, one v_cvt_pk_bf16_f32 (converting each half on its own
// costs two conversions plus a shift and an or)
__device__ inline uint32_t pack_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){lo, hi}, bf16x2_t));
}

// the same in the type DT
template <int DT>
__device__ inline uint32_t pack16x2(float lo, float hi) {
  if constexpr (DT == QW_DT_BF16) {
    return pack_bf16x2(lo, hi);
  } else {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){lo, hi}, f16x2));
  }
}
template <int DT>
__device__ inline floatx16 mma32(bf16x8 a, bf16x8 b, floatx16 c) {
  if constexpr (DT == QW_DT_BF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  } else {
    typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
}

// ---------------------------------------------------------------------------
// Prefill GEMM without anchor columns: W never goes through LDS.
//
// The four waves of a 256-thread workgroup each own 64 columns (two 32-wide
// sub-tiles) and all 256 rows of the 256 x 256 output tile (4 x ... = 8 x 2
// blocks of v_mfma_f32_32x32x16_bf16, 256 fp32 accumulators per lane). Each
// lane loads the packed codes and scales of its two columns for the next K
// step itself and dequantizes the B fragments (8 consecutive k of one
// column) in registers right before the products that use them, so every
// weight is dequantized once per workgroup and W costs no LDS traffic; only
// X is staged through two LDS buffers. The K loop is unrolled by two so the
// two register sets of W (current step, next step) have static indices.

// 8 consecutive bf16 weights (elements 8h..8h+7 of code dword c, element
// 16u + i in bits 2i..2i+1) from the packed value table T1:T0 of their group.
__device__ inline void dequant8_2bit(uint32_t c, int h, uint32_t T0, uint32_t T1, uint32_t out[4]) {
  const uint32_t cc = c >> (16 * h);
  uint32_t d[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) d[t] = (cc >> (2 * t)) & 0x00030303u;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int j = p >> 1, t = 2 * (p & 1);
    const uint32_t gsel = (uint32_t)j * 0x0101u + (uint32_t)(4 + j) * 0x01010000u;
    const uint32_t r = __builtin_amdgcn_perm(d[t + 1], d[t], gsel);  // q0 q0 q1 q1
    out[p] = __builtin_amdgcn_perm(T1, T0, (r << 1) + 0x01000100u);
  }
}

// Tile of workgroup b for an mt x nt grid of output tiles, XCD-aware.
// Workgroups are dealt to the 8 XCDs round-robin (b % 8), each XCD with its
// own L2. The q-th workgroup of XCD x takes tile t = (start of x's share) + q
// of an order that walks groups of up to 4 row tiles column by column, so
// the workgroups one XCD runs at a time cover a few row tiles times several
// column tiles: each W column tile is fetched once per XCD for the row tiles
// sharing it, instead of once per row tile (row tiles on different XCDs).
// A bijection for every grid size.
__device__ inline void xcd_tile(int b, int mt, int nt, int gmax, int &m_tile, int &n_tile) {
  if (gmax <= 0) {  // plain order: row tile fastest
    m_tile = b % mt;
    n_tile = b / mt;
    return;
  }
  constexpr int kXcds = 8;
  const int total = mt * nt;
  const int xcd = b % kXcds, q = b / kXcds;
  const int per = total / kXcds, rem = total % kXcds;
  const int t = xcd < rem ? xcd * (per + 1) + q : rem * (per + 1) + (xcd - rem) * per + q;
  const int gm = mt < gmax ? mt : gmax;   // row tiles per group
  const int g = t / (gm * nt);            // group of row tiles
  const int rows_g = min(gm, mt - g * gm);  // the last group may be narrower
  const int w = t - g * gm * nt;
  m_tile = g * gm + w % rows_g;
  n_tile = w / rows_g;
}

__device__ inline __amdgpu_buffer_rsrc_t pf_rsrc(const void *p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}
// An offset past every buffer's end (reads 0, drops stores): callers take
// these kernels only where X, Y and the codes are below so many bytes.
constexpr uint32_t kPfOob = 0x80000000u;

// Dynamic LDS bytes of a workgroup of four waves: two X buffers, over which
// the epilogue's slabs lie.
constexpr int prefill_w_lds(int rows, int nj) {
  const int x = 2 * rows * LDA * 2, slabs = 4 * 32 * (32 * nj + 4) * 4;
  return x > slabs ? x : slabs;
}

template <int FMT, bool F32OUT, int NJ, int WM, class Args>
__global__ __launch_bounds__(256 * WM) void prefill_w_kernel(Args a) {
  constexpr int BM = Args::kRows, DT = Args::kType;
  constexpr int NTW = 256 * WM;  // threads: WM x 4 waves
  constexpr int IM = BM / 32 / WM;  // 32-row blocks per wave
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];  // X [BM][LDA] x 2 buffers
  // NF4 level pairs (L[lo], L[hi]) of each code byte v, 16 replicas: replica r
  // of entry v at byte 256 v + 8 r, in bank pair r. Lane l reads replica
  // l % 16, so the table reads of 16 lanes never share a bank whatever the
  // codes (one 256-entry copy would collide about 3.5 ways per access).
  // (NF4 only: 2-bit and INT4 fragments are built from registers alone)
  constexpr bool kTab = FMT == QW_FMT_NF4_B64;
  // Entries lie 256 bytes apart, so that one byte permute makes an address;
  // tiles of 128 rows pack them (one more instruction) for two workgroups a CU.
  constexpr int kEntryBytes = BM > 128 ? 256 : 128;
  constexpr int kTabBytes = kTab ? 256 * kEntryBytes : 16;
  // fp16 operands: a column's weights enter times a power of two that brings
  // the largest that its scales allow to 2^14..2^15, and its sums leave
  // divided by it. fp16 by itself would hold neither a weight beyond 65504
  // nor, to its 11 bits, one below 2^-14; so it holds those down to 2^-28 of
  // the column's largest. bf16 has the exponents of fp32 and takes them as
  // they are. The scales are read twice for it (8192 fp16 rows over 8 experts
  // of 14336 x 4096 in 2-bit: 1148 us, 1072 without).
  constexpr bool kFit = DT == QW_DT_F16;
  __shared__ __attribute__((aligned(16))) char pair_tab[kTabBytes + (kFit ? 4 * 32 * NJ * 4 : 0)];
  const uint32_t lane_rep = 8u * (uint32_t)(threadIdx.x & 15);

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv >> 2, wn = wv & 3;  // wave's row half (WM = 2) and column quarter
  int m_tile, n_tile;
  RowTile rt{0, 0, 0};
  [[maybe_unused]] const uint32_t *codes = a.codes;  // of the tile's expert
  [[maybe_unused]] const void *scales = a.scales;
  if constexpr (Args::kGrouped) {
    const int row_tiles = count_row_tiles(a.offsets, a.G, a.n, BM);
    if ((int)blockIdx.x >= row_tiles * a.n_tiles) return;
    xcd_tile((int)blockIdx.x, row_tiles, a.n_tiles, a.xcd_group, m_tile, n_tile);
    rt = find_row_tile(a.offsets, a.G, a.n, BM, m_tile);
    // past an expert's rows a tile holds zeros, as past M
    const size_t weights = (size_t)rt.g * a.N * a.K;
    codes += FMT == QW_FMT_2BIT_G32 ? weights / 16 : weights / 8;
    scales = reinterpret_cast<const char *>(scales) + (FMT == QW_FMT_2BIT_G32 ? weights / 8 : weights / 16);
  } else {
    xcd_tile((int)blockIdx.x, a.mt_count, (int)gridDim.x / a.mt_count, a.xcd_group, m_tile, n_tile);
  }
  const int m0 = m_tile * BM, n0 = a.n_begin + n_tile * (128 * NJ);
  const int K = a.K;
  const int KT = K / BK;
  const int hk = lane >> 5;  // which 8 of each 16-wide k slice this lane holds

  if (kTab) {
    // 16-byte chunk c holds two replicas of entry c / 8
    for (int c = tid; c < 256 * 8; c += NTW) {
      const int v = c >> 3;
      const float2 p = make_float2(a.nf4[v & 15], a.nf4[v >> 4]);
      *reinterpret_cast<float4 *>(pair_tab + v * kEntryBytes + (c & 7) * 16) = make_float4(p.x, p.y, p.x, p.y);
    }
  }

  // ---- X prefetch registers (IM x 16 bytes per thread per step) ----
  // thread t copies 16-byte piece (t & 7) of rows (t >> 3) + 32 WM i, i < IM
  // (buffer loads: rows past M read through an out-of-range offset as 0)
  u32x4 ra[IM];
  const int xr = tid >> 3, xc = (tid & 7) * 8;
  const auto rx = pf_rsrc(a.X, (uint32_t)((size_t)a.M * K * 2));
  uint32_t xo[IM];
#pragma unroll
  for (int i = 0; i < IM; ++i) {
    int gm = m0 + xr + 32 * WM * i;
    if constexpr (Args::kGrouped) {
      const int q = xr + 32 * WM * i, p = rt.p0 + q;
      gm = q < rt.cnt ? (a.x_div ? x_row(a.rows[p], a.x_div, a.M) : p) : a.M;
      if (gm < 0) gm = a.M;
    }
    xo[i] = gm < a.M ? (uint32_t)(((size_t)gm * K + xc) * 2) : kPfOob;
  }
  // tiles at or past KT read as zeros (see the K loop below)
  auto load_x = [&](int kt) {
    const bool live = kt < KT;
    const uint32_t k0b = live ? (uint32_t)kt * BK * 2 : 0u;
#pragma unroll
    for (int i = 0; i < IM; ++i)
      ra[i] = __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(live ? xo[i] : kPfOob), (int)k0b, 0);
  };
  uint16_t *const xs = smem + xr * LDA + xc;  // + buf * BM * LDA + 32 WM i * LDA
  auto store_x = [&](int buf) {
#pragma unroll
    for (int i = 0; i < IM; ++i)
      *reinterpret_cast<u32x4 *>(xs + buf * BM * LDA + 32 * WM * i * LDA) = ra[i];
  };

  // ---- W registers of this lane's two columns, two sets (step parity) ----
  constexpr int WR = FMT == QW_FMT_2BIT_G32 ? 6 : 9;  // dwords per column per step
  uint32_t wr[2][NJ][WR];
  int gcol[NJ];
  bool cvalid[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    gcol[j] = n0 + wn * 32 * NJ + j * 32 + (lane & 31);
    cvalid[j] = gcol[j] < a.N;
  }
  const uint32_t cb = FMT == QW_FMT_2BIT_G32 ? (uint32_t)K / 4 : (uint32_t)K / 2;  // code bytes per column
  const uint32_t sb = FMT == QW_FMT_2BIT_G32 ? (uint32_t)K / 8 : (uint32_t)K / 16;  // scale bytes per column
  const auto rcode = pf_rsrc(Args::kGrouped ? codes : a.codes, (uint32_t)((size_t)a.N * cb));
  const auto rscale = pf_rsrc(Args::kGrouped ? scales : a.scales, (uint32_t)((size_t)a.N * sb));
  uint32_t co[NJ], so[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    co[j] = cvalid[j] ? (uint32_t)gcol[j] * cb : kPfOob;
    so[j] = cvalid[j] ? (uint32_t)gcol[j] * sb : kPfOob;
  }
  auto load_w = [&](int kt, uint32_t (&dst)[NJ][WR]) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (FMT == QW_FMT_2BIT_G32) {
        // 64 codes = 16 bytes, two S/Z words
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rcode, (int)co[j], kt * 16, 0);
          const u32x2 sz = __builtin_amdgcn_raw_buffer_load_b64(rscale, (int)so[j], kt * 8, 0);
        dst[j][0] = v[0]; dst[j][1] = v[1]; dst[j][2] = v[2]; dst[j][3] = v[3];
        dst[j][4] = sz[0]; dst[j][5] = sz[1];
      } else {
        // 64 codes = 32 bytes, one absmax
        const u32x4 v0 = __builtin_amdgcn_raw_buffer_load_b128(rcode, (int)co[j], kt * 32, 0);
        const u32x4 v1 = __builtin_amdgcn_raw_buffer_load_b128(rcode, (int)co[j], kt * 32 + 16, 0);
        dst[j][0] = v0[0]; dst[j][1] = v0[1]; dst[j][2] = v0[2]; dst[j][3] = v0[3];
        dst[j][4] = v1[0]; dst[j][5] = v1[1]; dst[j][6] = v1[2]; dst[j][7] = v1[3];
        dst[j][8] = __builtin_amdgcn_raw_buffer_load_b32(rscale, (int)so[j], kt * 4, 0);
      }
    }
  };

  [[maybe_unused]] float fit[NJ];  // the columns' powers of two
  [[maybe_unused]] float *const unfit = reinterpret_cast<float *>(pair_tab + kTabBytes) + wn * 32 * NJ;  // their inverses
  if constexpr (kFit) {
    // lanes l and l + 32 share a column and take its steps in turn
    float top[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) top[j] = 0.0f;
#pragma unroll 8
    for (int kt = hk; kt < KT; kt += 2) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        if (FMT == QW_FMT_2BIT_G32) {
          const u32x2 sz = __builtin_amdgcn_raw_buffer_load_b64(rscale, (int)(so[j] + (uint32_t)kt * 8), 0, 0);
#pragma unroll
          for (int g = 0; g < 2; ++g)
            top[j] = fmaxf(top[j], __builtin_fmaf(1.52f, fabsf(f16_bits_to_f32((uint16_t)sz[g])),
                                                  fabsf(f16_bits_to_f32((uint16_t)(sz[g] >> 16)))));
        } else {
          const uint32_t s = __builtin_amdgcn_raw_buffer_load_b32(rscale, (int)(so[j] + (uint32_t)kt * 4), 0, 0);
          if (FMT == QW_FMT_INT4_G32)
            top[j] = fmaxf(top[j], 8.0f * fmaxf(fabsf(f16_bits_to_f32((uint16_t)s)), fabsf(f16_bits_to_f32((uint16_t)(s >> 16)))));
          else
            top[j] = fmaxf(top[j], fabsf(__builtin_bit_cast(float, s)));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const float t = fmaxf(top[j], __shfl_xor(top[j], 32, 64));
      // 2^(14 - exponent of t), within what has a normal inverse; a column of
      // zeros, or with an infinite scale, as it is
      const int e = (int)(__builtin_bit_cast(uint32_t, t) >> 23) - 127;
      const int up = t > 0.0f && e < 128 ? min(14 - e, 126) : 0;
      fit[j] = __builtin_bit_cast(float, (uint32_t)(127 + up) << 23);
      unfit[j * 32 + (lane & 31)] = __builtin_bit_cast(float, (uint32_t)(127 - up) << 23);
    }
  }

  floatx16 acc[IM][NJ];
#pragma unroll
  for (int i = 0; i < IM; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  const uint16_t *const ar = smem + (wm * (BM / WM) + (lane & 31)) * LDA + hk * 8;  // + buf, i, kk offsets
  auto read_a = [&](int buf, int kk, bf16x8 (&af)[IM]) {
#pragma unroll
    for (int i = 0; i < IM; ++i)
      af[i] = *reinterpret_cast<const bf16x8 *>(ar + buf * BM * LDA + 32 * i * LDA + kk * 16);
  };

  // B fragment of column j for k slice kk of the step held in w
  auto make_b = [&](const uint32_t (&w)[NJ][WR], int j, int kk, const uint32_t (&T)[NJ][2][2]) {
    uint32_t o[4];
    if (FMT == QW_FMT_2BIT_G32) {
      const int g = kk >> 1;
      dequant8_2bit(w[j][kk], hk, T[j][g][0], T[j][g][1], o);
    } else if (FMT == QW_FMT_INT4_G32) {
      // the fp16 scale s of group kk / 2; elements kk*16 + hk*8 .. +7 are
      // the nibbles of code word 2kk + hk, element 2q in the low nibble of
      // byte q. Each nibble u becomes a float exactly (byte to float), and
      // u s - 8 s = (u - 8) s exactly (both products fit fp32), so the fma
      // gives fl32(s q) before the one rounding to bf16.
      float s = f16_bits_to_f32((uint16_t)(w[j][8] >> (16 * (kk >> 1))));
      if constexpr (kFit) s *= fit[j];
      const float ns8 = -8.0f * s;
      // the word picked with a byte permute (a select here becomes an
      // indexed read that moves the W registers to private memory)
      const uint32_t c = __builtin_amdgcn_perm(w[j][2 * kk + 1], w[j][2 * kk], hk ? 0x07060504u : 0x03020100u);
      const uint32_t lo = c & 0x0F0F0F0Fu, hi = (c >> 4) & 0x0F0F0F0Fu;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = pack16x2<DT>(__builtin_fmaf((float)((lo >> (8 * q)) & 0xFFu), s, ns8),
                           __builtin_fmaf((float)((hi >> (8 * q)) & 0xFFu), s, ns8));
    } else {
      // NF4: one fp32 absmax per 64
      float am = __builtin_bit_cast(float, w[j][8]);
      if constexpr (kFit) am *= fit[j];
      // elements kk*16 + hk*8 .. +7 = bytes 4*(2kk+hk) .. +3 of the 32 code bytes
      const uint32_t c = hk ? w[j][2 * kk + 1] : w[j][2 * kk];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // v_perm: byte 0 <- lane_rep (source byte 4), byte 1 <- code byte q
        const uint32_t ad = kEntryBytes == 256 ? __builtin_amdgcn_perm(lane_rep, c, 0x0C0C0004u | ((uint32_t)q << 8))
                                               : ((((c >> (8 * q)) & 0xFFu) << 7) | lane_rep);
        const float2 l = *reinterpret_cast<const float2 *>(pair_tab + ad);
        o[q] = pack16x2<DT>(am * l.x, am * l.y);
      }
    }
    return __builtin_bit_cast(bf16x8, u32x4{o[0], o[1], o[2], o[3]});
  };

  // One K step with the W register set PAR: products of tile kt out of LDS
  // buffer kt & 1; X of tile kt+1 is written to the other buffer after the
  // first k slice (the second for 2-bit), X of tile kt+2 and W of tile kt+1
  // (into the other set) are requested then too. W loads past the end re-read the last tile;
  // X loads past the end give zeros.
  // value tables of the two groups of each column (2-bit) from a W set
  auto make_tables = [&](const uint32_t (&w)[NJ][WR], uint32_t (&T)[NJ][2][2]) {
    if (FMT == QW_FMT_2BIT_G32) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t szw = w[j][4 + g];
          float S = f16_bits_to_f32((uint16_t)(szw & 0xFFFFu));
          float Z = f16_bits_to_f32((uint16_t)(szw >> 16));
          if constexpr (kFit) {
            S *= fit[j];
            Z *= fit[j];
          }
          T[j][g][0] = pack16x2<DT>(__builtin_fmaf(S, -1.52f, Z), __builtin_fmaf(S, -0.45f, Z));
          T[j][g][1] = pack16x2<DT>(__builtin_fmaf(S, 0.45f, Z), __builtin_fmaf(S, 1.52f, Z));
        }
    }
  };
  // 2-bit and INT4: the first slice's B fragments of a step (and the 2-bit
  // tables) depend on the lane's own W registers only, so they are built
  // during the previous step's last slice: after the step barrier only the
  // A reads remain before the first products (measured 3.6% faster for
  // 2-bit; NF4, whose fragments read the LDS pair table, keeps building
  // them at the step start: 30% slower otherwise).
  uint32_t T[NJ][2][2];
  bf16x8 fb0[NJ];

  auto step = [&](int kt, auto par_tag) {
    constexpr int PAR = decltype(par_tag)::value;
    constexpr int buf = PAR;  // kt has the parity of the register set
    const int kn1 = min(kt + 1, KT - 1), kn2 = kt + 2;
    // software pipeline: the A fragments and B fragments of slice kk+1 are
    // read and dequantized while the 16 products of slice kk run
    bf16x8 fa[2][IM], fb[2][NJ];
    read_a(buf, 0, fa[0]);
#pragma unroll
    for (int j = 0; j < NJ; ++j) fb[0][j] = !kTab ? fb0[j] : make_b(wr[PAR], j, 0, T);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk) {
      if (kk + 1 < BK / 16) {
        read_a(buf, kk + 1, fa[(kk + 1) & 1]);
#pragma unroll
        for (int j = 0; j < NJ; ++j) fb[(kk + 1) & 1][j] = make_b(wr[PAR], j, kk + 1, T);
      } else if constexpr (!kTab) {  // the next step's (W of tile kt+1)
        make_tables(wr[PAR ^ 1], T);
#pragma unroll
        for (int j = 0; j < NJ; ++j) fb0[j] = make_b(wr[PAR ^ 1], j, 0, T);
      }
#pragma unroll
      for (int i = 0; i < IM; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          acc[i][j] = mma32<DT>(fa[kk & 1][i], fb[kk & 1][j], acc[i][j]);
      // 2-bit: the next step's W is requested before X (so waiting for it
      // at the next step's start does not wait for X), and X is stored and
      // refilled one slice later (its wait overlaps a slice of products);
      // measured 2% faster for 2-bit, not for the 4-bit formats
      if constexpr (!kTab) {
        if (kk == 0) load_w(kn1, wr[PAR ^ 1]);
        if (kk == 1) {
          store_x(buf ^ 1);
          load_x(kn2);
        }
      } else if (kk == 0) {
        store_x(buf ^ 1);
        load_x(kn2);
        load_w(kn1, wr[PAR ^ 1]);
      }
      // IM NJ x {1 product, a few vector ops, a fragment read, an LDS write,
      // a memory read}: the vector work runs while the products execute
#pragma unroll
      for (int t = 0; t < IM * NJ; ++t) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);  // VALU
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // DS read
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // DS write
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // VMEM read
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // LDS-only barrier: the loads of the next steps stay in flight
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  };

  // prologue: X of tile 0 into buffer 0, X of tile 1 in registers, W of
  // tile 0 in set 0
  load_x(0);
  load_w(0, wr[0]);
  __syncthreads();  // the NF4 table too
  store_x(0);
  load_x(1);
  if constexpr (!kTab) {
    make_tables(wr[0], T);
#pragma unroll
    for (int j = 0; j < NJ; ++j) fb0[j] = make_b(wr[0], j, 0, T);
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  // Two steps per trip and a single exit: with an odd KT the last trip's
  // second step multiplies a zero X tile (one wasted step) rather than being
  // skipped, because a second loop exit makes the compiler copy the
  // accumulators out of the matrix-core registers on each path and spill.
  for (int kt = 0; kt < KT; kt += 2) {
    step(kt, std::integral_constant<int, 0>{});
    step(kt + 1, std::integral_constant<int, 1>{});
  }

  // ---- epilogue: lane holds D[8*g + 4*(lane>>5) + r][lane & 31] of each
  //      32 x 32 block. Each wave passes its 32 x 64 slice of one row block
  //      at a time through its own LDS slab (the X buffers are free now):
  //      accumulators go out with ds_write straight from the accumulator
  //      registers, come back as rows, and leave as 16-byte stores when the
  //      row length allows it (one element at a time otherwise). Buffer
  //      stores drop rows past M and columns past N. ----
  const uint32_t esz = F32OUT ? 4u : 2u;
  int y_rows = a.M;
  if constexpr (Args::kGrouped) y_rows = a.n;
  const auto ry = pf_rsrc(a.Y, (uint32_t)((size_t)y_rows * a.N * esz));
  constexpr int SL = 32 * NJ + 4;  // floats per slab row
  float *const slab = reinterpret_cast<float *>(smem) + wv * 32 * SL;
  const bool vec = F32OUT ? (a.N % 4 == 0) : (a.N % 8 == 0);
  // read-back mapping: CW columns per lane, RP rows per pass
  constexpr int CW = F32OUT ? 4 : 8;
  constexpr int LPR = 32 * NJ / CW;  // lanes per slab row
  constexpr int RP = 64 / LPR;
  // all lane-dependent epilogue addresses come from a copy of the lane index
  // the compiler cannot see through, so none of them is hoisted above the K
  // loop (where they would hold registers the whole time)
  int ln = lane;
  asm volatile("" : "+v"(ln));
  const int rr0 = ln / LPR, cc = (ln % LPR) * CW;
  // LDS byte address of this lane's first write: row 4 * (lane >> 5), column lane & 31
  const uint32_t slab_w = (uint32_t)reinterpret_cast<uintptr_t>(slab) +
                          (uint32_t)((4 * (ln >> 5) * SL + (ln & 31)) * 4);
  const int gc = n0 + wn * 32 * NJ + cc;
  static_assert(4 * WM * 32 * SL * 4 <= prefill_w_lds(BM, NJ), "slabs fit in the X buffers");
#pragma unroll
  for (int i = 0; i < IM; ++i) {
    // ds_write with the accumulator register as data operand: a plain store
    // makes the compiler copy acc to vector registers first, and that copy
    // pushes the allocator into spilling inside the K loop
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          asm volatile("ds_write_b32 %0, %1 offset:%2"
                       :
                       : "v"(slab_w), "a"(acc[i][j][4 * g + r]), "i"(((8 * g + r) * SL + j * 32) * 4)
                       : "memory");
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
#pragma unroll
    for (int pass = 0; pass < 32 / RP; ++pass) {
      const int rr = pass * RP + rr0;
      int gm = m0 + wm * (BM / WM) + i * 32 + rr;
      if constexpr (Args::kGrouped) {
        const int q = wm * (BM / WM) + i * 32 + rr, p = rt.p0 + q;
        gm = y_rows;
        if (q < rt.cnt) {
          gm = a.by_slot ? a.rows[p] : p;
          if (gm < 0 || (!a.by_slot && a.x_div && x_row(a.rows[p], a.x_div, a.M) < 0)) gm = y_rows;
        }
      }
      float v[CW];
#pragma unroll
      for (int q = 0; q < CW; q += 4) {
        const float4 t = *reinterpret_cast<const float4 *>(slab + rr * SL + cc + q);
        v[q] = t.x; v[q + 1] = t.y; v[q + 2] = t.z; v[q + 3] = t.w;
        if constexpr (kFit) {
          const float4 u = *reinterpret_cast<const float4 *>(unfit + cc + q);
          v[q] *= u.x; v[q + 1] *= u.y; v[q + 2] *= u.z; v[q + 3] *= u.w;
        }
      }
      const uint32_t rowb = gm < y_rows ? (uint32_t)gm * a.N * esz : kPfOob;
      if (vec) {
        const uint32_t off = (rowb != kPfOob && gc < a.N) ? rowb + (uint32_t)gc * esz : kPfOob;
        if (F32OUT) {
          const u32x4 o = {__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]),
                           __builtin_bit_cast(uint32_t, v[2]), __builtin_bit_cast(uint32_t, v[3])};
          __builtin_amdgcn_raw_buffer_store_b128(o, ry, (int)off, 0, 0);
        } else {
          const u32x4 o = {pack16x2<DT>(v[0], v[1]), pack16x2<DT>(v[2], v[3]),
                           pack16x2<DT>(v[4], v[5]), pack16x2<DT>(v[6], v[7])};
          __builtin_amdgcn_raw_buffer_store_b128(o, ry, (int)off, 0, 0);
        }
      } else {
#pragma unroll
        for (int q = 0; q < CW; ++q) {
          const uint32_t off =
              (rowb != kPfOob && gc + q < a.N) ? rowb + (uint32_t)(gc + q) * esz : kPfOob;
          if (F32OUT)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v[q]), ry, (int)off, 0, 0);
          else
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)Op<DT>::bits(v[q]), ry, (int)off, 0, 0);
        }
      }
    }
    // the slab is rewritten by the next row block
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  }
}

}  // namespace
}  // namespace qw
