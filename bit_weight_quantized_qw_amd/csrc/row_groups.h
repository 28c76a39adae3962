// Rows grouped by the matrix they take (qw_groups): the device-side lookup
// shared by the kernels that walk tiles of grouped rows.
#pragma once

#include "qw_internal.h"

namespace qw {

// One tile of up to `height` rows of one group.
struct RowTile {
  int g;    // group
  int p0;   // first position
  int cnt;  // rows in the tile, 1..height; 0: there is no such tile
};

// Tile number `tile` of the tiles that cut every group into runs of up to
// `height` positions, groups in order. Called by whole waves with
// wave-uniform arguments; the result is wave-uniform. The offsets are
// clamped to 0..n and a descending pair counts as an empty group, so the
// positions of a tile lie in 0..n-1 whatever the arrays hold. With `rest`
// the positions behind the last group count as one more group, number G.
// 64 groups a step, one load behind another: 16 rows of the last of 64
// experts of 512 x 512 5.4 us, of 256 6.7, of 1024 11.7.
__device__ inline RowTile find_row_tile(const int32_t *offsets, int G, int n, int height, int tile,
                                        bool rest = false) {
  const int lane = threadIdx.x & 63;
  const int groups = rest ? G + 1 : G;
  int before = 0;  // tiles of the groups before this run of 64
  for (int g0 = 0; g0 < groups; g0 += 64) {
    const int g = g0 + lane;
    int lo = 0, hi = 0;
    if (g < groups) {
      lo = min(max(offsets[g], 0), n);
      hi = g < G ? min(max(offsets[g + 1], lo), n) : n;
    }
    const int own = (hi - lo + height - 1) / height;
    int upto = own;  // inclusive prefix sum over the wave
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    const uint64_t past = __ballot(before + upto > tile);
    if (past) {
      const int f = __ffsll((unsigned long long)past) - 1;
      const int first = before + __builtin_amdgcn_readlane(upto, f) - __builtin_amdgcn_readlane(own, f);
      const int p0 = __builtin_amdgcn_readlane(lo, f) + (tile - first) * height;
      const int end = __builtin_amdgcn_readlane(hi, f);
      return RowTile{g0 + f, p0, min(height, end - p0)};
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return RowTile{0, 0, 0};
}

// rows[] by position. Few rows are read at once, one a lane, before the
// position is known: a short launch is a chain of dependent loads from cold
// memory (a microsecond each), of which this takes one out. Made and asked
// by whole waves; p must be in 0..n-1.
struct RowLookup {
  const int32_t *rows;
  bool small;
  int mine;
  __device__ RowLookup(const int32_t *r, int n) : rows(r), small(n <= 64), mine(0) {
    if (small) mine = r[min((int)(threadIdx.x & 63), n - 1)];
  }
  __device__ int operator()(int p) const { return small ? __shfl(mine, p, 64) : rows[p]; }
};

// The row of X that row number r takes, r / x_div; -1 where r is out of range
// (the quotient alone would take -1 for row 0).
__device__ inline int x_row(int r, int x_div, int x_rows) {
  const int q = r / x_div;
  return r >= 0 && q < x_rows ? q : -1;
}

// Number of those tiles, wave-uniform; no more than ascending offsets can
// make (what the grid was sized for), whatever the offsets are.
__device__ inline int count_row_tiles(const int32_t *offsets, int G, int n, int height) {
  int own = 0;
  for (int g = threadIdx.x & 63; g < G; g += 64) {
    const int lo = min(max(offsets[g], 0), n);
    own += (min(max(offsets[g + 1], lo), n) - lo + height - 1) / height;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) own += __shfl_xor(own, d, 64);
  return min(__builtin_amdgcn_readfirstlane(own), n / height + G);
}

// Most tiles that n rows in G groups can make: every group ends in at most
// one short tile, and no tile is empty.
inline long long most_row_tiles(int n, int G, int height) {
  const long long full = (long long)n / height + G;
  return full < n ? full : n;
}

// Most workgroups of one launch, all of which have 256 threads here: a
// dispatch counts its threads in 32 bits.
constexpr long long kMostBlocks = (1ll << 24) - 1;

// Validates a qw_groups view (sizes, NULLs, alignment).
inline qw_status check_groups(const qw_groups *g) {
  if (!g || g->G < 1 || g->n < 1 || !g->offsets || !g->rows) return QW_ERR_INVALID_ARG;
  if (!aligned16(g->offsets) || !aligned16(g->rows)) return QW_ERR_ALIGNMENT;
  if (g->G > QW_MAX_GROUPS || g->n > QW_MAX_ROWS) return QW_ERR_UNSUPPORTED;
  return QW_OK;
}

}  // namespace qw
