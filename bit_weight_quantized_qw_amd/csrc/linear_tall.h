// The products of qgemm_linear by tall tiles, for many rows: the prefill GEMM's
// kernel (prefill_w.h) with 8-bit activations, fp16 anchors, K in parts and
// what stands behind the sums.
#pragma once

#include "prefill_w.h"

namespace qw {
namespace {

// Columns n_begin .. n_begin + columns of Y, by tiles of ROWS rows.
template <int FMT, int ROWS, int XT, bool MASK, bool GATED>
qw_status launch_columns(const LinearArgs &l, int n_begin, int columns, hipStream_t s) {
  if (columns <= 0) return QW_OK;
  using Args = LinearTallArgs<ROWS, XT, MASK, GATED>;
  constexpr auto kernel = prefill_w_kernel<FMT, true, 2, 1, Args>;
  const size_t lds = prefill_w_lds(ROWS, 2);
  QW_HIP_TRY(hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds));
  Args a{};
  a.codes = reinterpret_cast<const uint32_t *>(l.codes);
  a.scales = l.scales;
  a.idx = l.idx;
  a.wo = l.wo;
  a.mask = l.mask;
  a.N = l.N;
  a.K = l.K;
  a.n_out = l.n_out;
  a.n_out_pad = l.n_out_pad;
  a.xcd_group = 4;
  for (int i = 0; i < 16; ++i) a.nf4[i] = l.nf4[i];
  a.n_begin = n_begin;
  a.n_tiles = (columns + tall_columns(GATED) - 1) / tall_columns(GATED);
  a.parts = l.parts;
  a.fin = l.fin;
  // offsets into X have 32 bits: as many rows a launch as lie below them
  const size_t row_bytes = (size_t)l.K * (Args::kIn8 ? 1 : 2);
  const long long by_bytes = (long long)((kPfOob - 1) / row_bytes) / ROWS * ROWS;
  const long long by_grid = kMostBlocks / ((long long)a.n_tiles * a.parts) * ROWS;
  const long long most = by_bytes < by_grid ? by_bytes : by_grid;
  if (most < ROWS) return QW_ERR_UNSUPPORTED;
  for (long long m = 0; m < l.M; m += most) {
    a.M = (int)(l.M - m < most ? l.M - m : most);
    a.m_first = (int)m;
    a.X = reinterpret_cast<const uint16_t *>(reinterpret_cast<const char *>(l.X) + (size_t)m * row_bytes);
    a.mt_count = (a.M + ROWS - 1) / ROWS;
    QW_HIP_TRY(launch(kernel, (unsigned)(a.mt_count * a.n_tiles * a.parts), 256, lds, s, a));
  }
  return QW_OK;
}

template <int FMT, int XT, bool MASK, bool GATED>
qw_status launch_tiles(const LinearArgs &a, int high_tiles, hipStream_t s) {
  const int most = (a.fin.out_n + tall_columns(GATED) - 1) / tall_columns(GATED) * tall_columns(GATED);
  const int high = high_tiles * tall_columns(GATED) < most ? high_tiles * tall_columns(GATED) : most;
  QW_TRY((launch_columns<FMT, 256, XT, MASK, GATED>(a, 0, high < a.fin.out_n ? high : a.fin.out_n, s)));
  return launch_columns<FMT, 128, XT, MASK, GATED>(a, high, a.fin.out_n - high, s);
}

template <int FMT, int XT, bool MASK>
qw_status launch_gated(const LinearArgs &a, int high_tiles, hipStream_t s) {
  return a.fin.gated ? launch_tiles<FMT, XT, MASK, true>(a, high_tiles, s) : launch_tiles<FMT, XT, MASK, false>(a, high_tiles, s);
}

template <int FMT, int XT>
qw_status launch_tall_type(const LinearArgs &a, int high_tiles, hipStream_t s) {
  if constexpr (FMT == QW_FMT_2BIT_G32)
    if (a.n_out > 0) return launch_gated<FMT, XT, true>(a, high_tiles, s);
  return launch_gated<FMT, XT, false>(a, high_tiles, s);
}

}  // namespace

template <int FMT>
qw_status launch_linear_tall(const LinearArgs &a, int high_tiles, hipStream_t s) {
  switch (a.x_dtype) {
    case QW_DT_F16: return launch_tall_type<FMT, QW_DT_F16>(a, high_tiles, s);
    case QW_DT_BF16: return launch_tall_type<FMT, QW_DT_BF16>(a, high_tiles, s);
    case QW_DT_E4M3: return launch_tall_type<FMT, QW_DT_E4M3>(a, high_tiles, s);
    default: return launch_tall_type<FMT, QW_DT_I8>(a, high_tiles, s);
  }
}

}  // namespace qw
