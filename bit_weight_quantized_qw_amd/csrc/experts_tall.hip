// The experts' products for many rows per expert: the prefill
// GEMM's kernel with its row tiles cut from the groups. The matrix cores
// bound it. Against the wide tiles the weights are scaled and rounded to
// X's type before the product, as in qgemm_prefill: scaling the fp32 sums costs
// a multiply-add per 32 products in vector units that, beside decoding, are
// then what bounds (8 experts of 14336 x 4096 in 2-bit, 8192 rows: 0.28 of
// the matrix cores' cycles there). That call here: 2-bit 950 us (fp16 1150),
// INT4 1050 (1130), NF4 1170 (1240).
//
// Anchors, gated products and rows or outputs of 2 GiB and more (byte offsets
// have 32 bits) go to the wide tiles, however many the rows: the same call
// with anchors takes 2140 us in 2-bit and 1600 in INT4; the sum of 8 of 16
// experts of 4096 x 1408 takes 2260 us for 15872 tokens in 2-bit and, its
// products past 2 GiB, 3380 for 16384.
#include "experts.h"
#include "prefill_w.h"

namespace qw {
namespace {

template <int FMT, bool F32, int ROWS, int DT>
qw_status launch_tall(const GroupedArgs<ROWS, DT> &a, hipStream_t s) {
  constexpr auto kernel = prefill_w_kernel<FMT, F32, 2, 1, GroupedArgs<ROWS, DT>>;
  const size_t lds = prefill_w_lds(ROWS, 2);
  const long long grid = most_row_tiles(a.n, a.G, ROWS) * a.n_tiles;
  if (grid > kMostBlocks) return QW_ERR_UNSUPPORTED;
  QW_HIP_TRY(hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds));
  QW_HIP_TRY(launch(kernel, (unsigned)grid, 256, lds, s, a));
  return QW_OK;
}

template <int FMT, int ROWS, int DT>
qw_status launch_type(const ExpertArgs &e, hipStream_t s) {
  GroupedArgs<ROWS, DT> a{};
  a.X = e.X;
  a.codes = reinterpret_cast<const uint32_t *>(e.codes);
  a.scales = e.scales;
  a.Y = e.Y;
  a.M = e.x_rows;
  a.N = e.N;
  a.K = e.K;
  a.xcd_group = 4;
  for (int i = 0; i < 16; ++i) a.nf4[i] = e.nf4[i];
  a.offsets = e.offsets;
  a.rows = e.rows;
  a.G = e.G;
  a.n = e.n;
  a.x_div = e.x_div;
  a.by_slot = e.by_slot;
  a.n_tiles = (e.N + 255) / 256;
  return e.y_dtype == QW_DT_F32 ? launch_tall<FMT, true, ROWS, DT>(a, s) : launch_tall<FMT, false, ROWS, DT>(a, s);
}

template <int ROWS, int DT>
qw_status launch_fmt(int fmt, const ExpertArgs &a, hipStream_t s) {
  if (fmt == QW_FMT_2BIT_G32) return launch_type<QW_FMT_2BIT_G32, ROWS, DT>(a, s);
  if (fmt == QW_FMT_INT4_G32) return launch_type<QW_FMT_INT4_G32, ROWS, DT>(a, s);
  return launch_type<QW_FMT_NF4_B64, ROWS, DT>(a, s);
}

}  // namespace

bool experts_tall_fits(int x_dtype, const ExpertArgs &a) {
  const size_t lim = kPfOob, esz = a.y_dtype == QW_DT_F32 ? 4 : 2;
  return (a.y_dtype == QW_DT_F32 || a.y_dtype == x_dtype) && !a.swiglu && a.n_out == 0 &&
         (size_t)a.x_rows * a.K * 2 < lim && (size_t)a.n * a.N * esz < lim;
}

qw_status launch_experts_tall(int fmt, int x_dtype, int row_blocks, const ExpertArgs &a, hipStream_t s) {
  if (x_dtype == QW_DT_F16)
    return row_blocks <= 8 ? launch_fmt<128, QW_DT_F16>(fmt, a, s) : launch_fmt<256, QW_DT_F16>(fmt, a, s);
  return row_blocks <= 8 ? launch_fmt<128, QW_DT_BF16>(fmt, a, s) : launch_fmt<256, QW_DT_BF16>(fmt, a, s);
}

}  // namespace qw
