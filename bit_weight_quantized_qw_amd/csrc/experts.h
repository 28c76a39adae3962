// What the experts' products share: their arguments, the lane exchanges that
// bring packed codes into operand order, and the table of code levels.
#pragma once

#include "op16.h"
#include "row_groups.h"

namespace qw {

struct ExpertArgs {
  const uint16_t *X;        // [x_rows][K]
  const uint8_t *codes;
  const uint8_t *scales;
  const int32_t *idx;       // 2-bit anchors [E][n_out]
  const uint32_t *mask;     // 2-bit anchors [E][K/32]
  const uint16_t *wo;       // anchors [E][N][n_out_pad], fp16
  const int32_t *offsets, *rows;
  void *Y;
  int x_rows, x_div;
  int G, n;                 // groups, positions
  int N, K, out_n;          // weight rows, weight columns, columns of Y
  int n_out, n_out_pad;
  int col_tiles;
  int swiglu, by_slot;      // by_slot: Y row rows[p] in place of p
  int y_dtype;
  float nf4[16];            // NF4 levels as the kernel's table takes them
  float level_unit;         // wide tiles: what one unit of them is worth
};

__device__ inline __amdgpu_buffer_rsrc_t rsrc(const void *p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}
constexpr uint32_t kOob = 0x80000000u;  // an offset past every buffer's end (reads 0)

__device__ inline void swap32(uint32_t &a, uint32_t &b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ inline void swap16(uint32_t &a, uint32_t &b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
// d[i] of lane group g (lanes 16g..16g+15) <-> d[g] of lane group i
__device__ inline void transpose4(uint32_t (&d)[4]) {
  swap32(d[0], d[2]);
  swap32(d[1], d[3]);
  swap16(d[0], d[1]);
  swap16(d[2], d[3]);
}
// w of lane group i to all four lane groups, as out[i]
__device__ inline void gather4(uint32_t w, uint32_t (&out)[4]) {
  uint32_t a = w, b = w;
  swap32(a, b);  // a: groups 0 1 0 1, b: groups 2 3 2 3
  out[0] = out[1] = a;
  out[2] = out[3] = b;
  swap16(out[0], out[1]);
  swap16(out[2], out[3]);
}

// w of lane group g (a constant) to all four lane groups
__device__ inline uint32_t from_group(uint32_t w, int g) {
  uint32_t a = w, b = w;
  swap32(a, b);  // a: groups 0 1 0 1, b: groups 2 3 2 3
  uint32_t c = g & 2 ? b : a, d = c;
  swap16(c, d);  // c: 0 0 0 0 (or 2 2 2 2), d: the odd one
  return g & 1 ? d : c;
}
// 2-bit: halves h0..h7 of a lane's 64 codes, so that dword g gets (h_g,
// h_4+g): after the transposition lane group g has its 8 codes of the steps
// 2s and 2s + 1 (32 weights each) in dword s
__device__ inline void to_halves(uint32_t (&d)[4]) {
  const uint32_t d0 = d[0], d1 = d[1], d2 = d[2], d3 = d[3];
  d[0] = __builtin_amdgcn_perm(d2, d0, 0x05040100u);
  d[1] = __builtin_amdgcn_perm(d2, d0, 0x07060302u);
  d[2] = __builtin_amdgcn_perm(d3, d1, 0x05040100u);
  d[3] = __builtin_amdgcn_perm(d3, d1, 0x07060302u);
}
// eight fp16 anchors as two bf16 numbers each (exactly: 8 + 3 bits)
__device__ inline void split_f16(u32x4 &b, u32x4 &rest) {
  using O = Op<QW_DT_BF16>;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float lo = f16_bits_to_f32((uint16_t)b[q]), hi = f16_bits_to_f32((uint16_t)(b[q] >> 16));
    const uint32_t lo16 = O::bits(lo), hi16 = O::bits(hi);
    b[q] = lo16 | (hi16 << 16);
    rest[q] = O::bits(lo - O::value(lo16)) | (O::bits(hi - O::value(hi16)) << 16);
  }
}

// A row tile and the column tile of one workgroup.
struct TileAt {
  RowTile rows;
  int col;
};

// Workgroup b's tile of row tiles x col_tiles. Workgroups go to the 8 XCDs
// in turn, each with an L2 of its own; so each XCD takes a run of the tiles
// in an order that walks up to 8 row tiles column by column: what it works
// on at a time shares its rows of X and its columns of W.
__device__ inline TileAt place_tile(const int32_t *offsets, int G, int n, int height, int col_tiles, int b) {
  const int row_tiles = count_row_tiles(offsets, G, n, height);
  const int total = row_tiles * col_tiles;  // the grid bounds it below 2^31
  if (b >= total) return TileAt{RowTile{0, 0, 0}, 0};
  const int xcd = b % 8, q = b / 8, per = total / 8, rem = total % 8;
  const int t = xcd * per + min(xcd, rem) + q;
  const int band = t / (8 * col_tiles), w = t - band * 8 * col_tiles;
  const int high = min(8, row_tiles - band * 8);
  return TileAt{find_row_tile(offsets, G, n, height, band * 8 + w % high), w / high};
}

// INT4 operands without a table: a nibble u put into the top mantissa bits
// of 16 is the number 16 + u, and two nibbles 16 bits apart are done at
// once. The elements of a word then come in the order 0 4 1 5 2 6 3 7, which
// the operand of X is brought into, and the products start from -24 times
// the row sums of x.
template <int DT>
struct Int4 {
  static constexpr int kAt = DT == QW_DT_F16 ? 6 : 3;  // where the top four mantissa bits begin
  static constexpr uint32_t kSixteen = (DT == QW_DT_F16 ? 0x4C00u : 0x4180u) * 0x10001u;
  static constexpr uint32_t kMinus24 = (DT == QW_DT_F16 ? 0xCE00u : 0xC1C0u) * 0x10001u;
  static __device__ u32x4 operand(uint32_t c, uint32_t sixteen) {
    constexpr uint32_t mask = 0x000F000Fu << kAt;
    u32x4 b;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int up = kAt - 4 * q;
      b[q] = ((up >= 0 ? c << (up & 31) : c >> (-up & 31)) & mask) | sixteen;
    }
    return b;
  }
  static __device__ u32x4 order(u32x4 x) {
    return u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                 __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
  }
};

// Level table: entry of code byte v, replica r. 2-bit: four levels (8
// bytes), wide NF4: two (4 bytes, two replicas side by side), narrow NF4:
// the nearest two and the rests of both (8 bytes).
constexpr int kEntry = 128;  // bytes of one byte's replicas
template <int FMT, int DT, int kThreads, bool WIDE = false>
__device__ inline void fill_table(char *tab, const ExpertArgs &a) {
  // one entry's value per thread, then its 128 bytes; neighbours start at
  // different pieces, so that they write different banks
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
    } else if (WIDE) {
      const uint32_t p = Op<DT>::bits(a.nf4[v & 15]) | (Op<DT>::bits(a.nf4[v >> 4]) << 16);
      w = u32x2{p, p};
    } else {
      const float lo = a.nf4[v & 15], hi = a.nf4[v >> 4];
      const uint32_t lo16 = Op<DT>::bits(lo), hi16 = Op<DT>::bits(hi);
      w = u32x2{lo16 | (hi16 << 16),
                Op<DT>::bits(lo - Op<DT>::value(lo16)) | (Op<DT>::bits(hi - Op<DT>::value(hi16)) << 16)};
    }
#pragma unroll
    for (int r = 0; r < 8; ++r)
      *reinterpret_cast<u32x4 *>(tab + v * kEntry + ((r + v) & 7) * 16) = u32x4{w[0], w[1], w[0], w[1]};
  }
}

// The products by tiles of 32 or 64 rows (experts_wide.hip).
qw_status launch_experts_wide(int fmt, int x_dtype, int row_blocks, const ExpertArgs &a, hipStream_t s);

// The products by tiles of 128 or 256 rows (experts_tall.hip), and whether
// that kernel takes the call: no anchors, not gated, Y of X's type or fp32,
// and the rows and outputs within 32-bit offsets.
bool experts_tall_fits(int x_dtype, const ExpertArgs &a);
qw_status launch_experts_tall(int fmt, int x_dtype, int row_blocks, const ExpertArgs &a, hipStream_t s);

}  // namespace qw
