// A packed matrix times any number of rows, with bias, activation, gate and
// residual applied to the fp32 sums:
//   Y[m][n] = act(x_scales[m] sum_k X[m][k] w[n][k] + bias[n]) + residual[m][n]
// The kernels are in linear_narrow.h (few rows) and linear_tall.h (many); here
// stand the choice between them and the sum over parts of K.
#include <math.h>

#include "linear.h"

namespace qw {
namespace {

// Adds up the parts of K in order, then what stands behind the sums. A thread
// takes four columns of a row.
__global__ __launch_bounds__(256) void join_kernel(Finish a, int parts, int col_blocks, int m_first) {
  const int m = m_first + (int)(blockIdx.x / col_blocks);
  const int n = ((int)(blockIdx.x % col_blocks) * 256 + (int)threadIdx.x) * 4;
  if (n >= a.out_n) return;
  const bool vec = a.out_n % 4 == 0;
  f32x4 s = {0, 0, 0, 0}, up = {0, 0, 0, 0};
  for (int p = 0; p < parts; ++p) {
    const size_t row = ((size_t)p * a.M + m) * a.N;
    s += load_four(a.partial, row + n, QW_DT_F32, a.out_n - n, vec);
    if (a.gated) up += load_four(a.partial, row + a.out_n + n, QW_DT_F32, a.out_n - n, vec);
  }
  store_four(a, m, n, shape_values(a, s, up, scale_at(a, m), bias_at(a, n), bias_up_at(a, n)) + residual_at(a, m, n));
}

// Rows of bf16 as rows of fp16 times a power of two a row, for gated products by
// tall tiles: rounded to bf16, the weights of gate and up would leave 1.7 times
// the error that Y's own rounding leaves (2.9e-3 against 1.7e-3 of Y, 2000 rows
// of 27648 x 5120 in INT4), rounded to fp16 they leave no more than it. A bf16
// number is an fp16 one from the row's largest down to 2^-28 of it. Bound by
// memory; a workgroup reads its row twice, the second time from the cache.
// Products that are not gated keep bf16 weights whatever Y's type: with a Y in fp16
// the weights are what is off then (434 rows of 7379 x 5440 in INT4 8.2e-4 of Y and
// an fp32 residual, 2.1e-4 from Y's rounding alone), and fp16 ones cost 8 to 12 % of
// prompts (2048 rows of 28672 x 8192 in 2-bit 913 and 1027 us) and up to a half of
// 100 rows (8192 x 28672 in 2-bit with anchors 94 and 140 us). Rows given in fp16
// have them.
__global__ __launch_bounds__(256) void to_fp16_kernel(const uint16_t *X, uint16_t *out, float *scales, int m_first, int K) {
  __shared__ uint32_t tops[4];
  const size_t m = (size_t)m_first + blockIdx.x;
  const u32x4 *from = reinterpret_cast<const u32x4 *>(X + m * K);
  uint32_t top = 0;  // the largest pattern without its sign
  for (int i = threadIdx.x; i < K / 8; i += 256) {
    const u32x4 v = from[i];
#pragma unroll
    for (int q = 0; q < 4; ++q) top = max(top, max(v[q] & 0x7FFFu, (v[q] >> 16) & 0x7FFFu));
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  // the largest to 2^14 .. 2^15 (beside an infinity or a NaN as beside the largest
  // number, so that no finite one becomes infinite), rows of zeros as they are
  const int e = min((int)(top >> 7) - 127, 127);
  const int up = top > 0 ? min(14 - e, 126) : 0;
  const float f = __builtin_bit_cast(float, (uint32_t)(127 + up) << 23);
  if (threadIdx.x == 0) scales[m] = __builtin_bit_cast(float, (uint32_t)(127 - up) << 23);
  u32x4 *to = reinterpret_cast<u32x4 *>(out + m * K);
  for (int i = threadIdx.x; i < K / 8; i += 256) {
    const u32x4 v = from[i];
    u32x4 w;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = Op<QW_DT_F16>::bits(__builtin_bit_cast(float, v[q] << 16) * f) |
             (Op<QW_DT_F16>::bits(__builtin_bit_cast(float, v[q] & 0xFFFF0000u) * f) << 16);
    to[i] = w;
  }
}

// How a call runs: a decode GEMV, the narrow kernel with tiles of `shape`, or the
// tall one, the first high_tiles tiles of columns with 256 rows; and the parts
// of K.
enum class Kernel { kGemv, kNarrow, kTall };
struct Plan {
  Kernel kernel;
  int shape, high_tiles, parts;
  bool to_fp16;  // bf16 activations, as fp16 ones
};

// Workspace: the parts' sums, then fp16 activations and their rows' scales.
size_t parts_bytes(const Plan &p, int M, int N) {
  return p.parts > 1 ? ((size_t)p.parts * M * N * sizeof(float) + 15) / 16 * 16 : 0;
}
size_t fp16_bytes(int M, int K) { return (size_t)M * K * 2; }
size_t workspace_of(const Plan &p, int M, int N, int K) {
  return parts_bytes(p, M, N) + (p.to_fp16 ? fp16_bytes(M, K) + (size_t)M * sizeof(float) : 0);
}

// Tile and waves of the narrow kernel for row blocks MR (0: up to four rows): as
// many workgroups and waves as fill the CUs, more columns a wave where there
// are enough of them (what a wave loads of X serves them all). With tiles of 32
// and 64 columns, 8 waves each, us: 16 rows of 5120 x 5120 in 2-bit 16.9 / 21.9,
// of 11008 x 4096 in NF4 19.1 / 16.4, of 27648 x 5120 in INT4 44.8 / 35.7. Tiles
// of four rows against sixteen, one row of 8192 x 28672: 2-bit 39 / 47, NF4 33 /
// 36, INT4 37 / 36 (so it has none).
int pick_narrow(int MR, int fmt, int out_n, int K, bool gated) {
  const int blocks = (out_n + 15) / 16 * (gated ? 2 : 1), chunks = (K + 255) / 256;
  if (MR == 0) {
    if (fmt == QW_FMT_INT4_G32) MR = 1;  // no quicker for it
  }
  if (MR == 0) {
    if (blocks <= 400 && !gated && chunks <= 48) return narrow_shape(0, 1, 8);
    const int waves = 4200 / (blocks / 2 + 1);
    return narrow_shape(0, 2, waves >= 16 ? 16 : waves >= 8 ? 8 : 4);
  }
  if (blocks < 600) return narrow_shape(MR, 2, 8);
  return narrow_shape(MR, 4, MR == 1 && blocks / 4 > 300 ? 4 : 8);
}

// Column tiles by 256 rows: whole rounds over the CUs, and the rest by tiles of
// 128 rows, two workgroups a CU, in place of a round that fills few of them.
// Times in rounds of high tiles; two low tiles side by side take 1.1 of one, a
// low tile alone 0.6.
int pick_high_tiles(int M, int nt) {
  const int high = (M + 255) / 256, low = (M + 127) / 128;
  double best = 1e30;
  int best_n = 0;
  for (int n = nt; n >= 0; --n) {
    const long long h = (long long)high * n, l = (long long)low * (nt - n);
    const double cost = (double)((h + 255) / 256) + (double)(l / 512) * 1.1 + (l % 512 == 0 ? 0.0 : l % 512 <= 256 ? 0.6 : 1.1);
    if (cost < best - 1e-9) {
      best = cost;
      best_n = n;
    }
  }
  return best_n;
}

// Estimated time of the tall kernel, us, with every column tile 256 (high) or
// 128 rows high and K in `parts`: a start, the steps of 64 elements one behind
// another, slower where two workgroups share a CU or follow each other, and the
// sum over the parts. A step of a workgroup alone on its CU is bound by the
// issue of its own waves (products, and decoding beside them), not by memory:
// loads three steps ahead instead of one left it as it was. And of the narrow
// kernel with tiles of 32 rows: what its products take. Measured / estimated
// (bf16; with anchors int8), M x N x K: narrow, and by 128 rows with K in 1, 4
// and 8 parts:
//   2-bit, anchors 100 x  5120 x  5120    70/83     108/114     40/43      31/33
//   2-bit, anchors 100 x  8192 x 28672   399/409    560/592    155/165     95/97
//   2-bit, anchors 333 x  1501 x  2048    36/32      59/52      33/27      35/25
//   2-bit          100 x  5120 x  5120    48/50      81/86      32/36      25/30
//   2-bit          100 x  8192 x 28672   253/309    389/436    115/125     77/77
//   2-bit          333 x  1501 x  2048    27/22      45/40      27/25      30/24
//   NF4            100 x  5120 x  5120    53/50     156/162     59/55      44/39
//   NF4            100 x  8192 x 28672   284/309    802/861    230/232    138/130
//   NF4            333 x  1501 x  2048    30/22      83/71      46/32      45/28
//   INT4           100 x  5120 x  5120    49/50     107/108     38/42      28/33
//   INT4           100 x  8192 x 28672   266/309    562/557    158/156     95/92
//   INT4           333 x  1501 x  2048    26/22      52/49      29/27      31/25
double tall_time(int fmt, bool anchors, int M, int nt, int N, int K, bool high, int parts) {
  const int f = fmt == QW_FMT_2BIT_G32 ? anchors : fmt == QW_FMT_NF4_B64 ? 2 : 3;
  constexpr double kStep[4][2] = {{0.95, 1.35}, {1.3, 1.9}, {1.9, 2.8}, {1.22, 1.65}};
  const double steps = ceil((double)(K / 64) / parts);
  const double groups = (double)((M + (high ? 255 : 127)) / (high ? 256 : 128)) * nt * parts;
  const double rounds = high ? ceil(groups / 256) : groups <= 256 ? 1.0 : 1.7 * fmax(1.0, groups / 512 + 0.2);
  return 10 + steps * kStep[f][high] * rounds + (parts > 1 ? 4 + 8.0 * parts * M * N / 5.2e6 : 0);
}
// A narrow grid of 256 workgroups and fewer is one round, whatever its rows: each
// of them passes through all of K. us, measured / estimated, narrow, and by 128 rows
// with K in 16 parts (bf16 rows, anchors with INT4):
//   2-bit           40 x 500 x  4096   16/17     16/18
//   2-bit           40 x 500 x  8192   25/25     19/22
//   2-bit          100 x 500 x 28672   70/68     38/42
//   NF4             40 x 500 x 11008   32/33     40/35
//   NF4             40 x 500 x 28672   75/74     67/67
//   INT4            40 x 500 x  4096   18/18     18/19
//   INT4            40 x 500 x  8192   27/28     23/24
//   INT4           100 x 500 x 28672   78/77     49/50
// 2-bit with anchors, bf16 rows and int8 rows, narrow, and in 16 parts: 4096 20 21,
// 20 23; 6144 25 25, 22 27; 8192 35 34, 24 30; 28672 106 96, 46 71 (40 rows of 500).
// A round takes 3.4e-3 a step of K there, and 2.4e-3 are counted: int8 rows take
// longer by tall tiles than is estimated, and between the two kinds' borders (5000
// and 7000) it is the narrow kernel that rounds no weight.
double narrow_time(int fmt, bool anchors, int M, int N, int K, int shape) {
  const int f = fmt == QW_FMT_2BIT_G32 ? anchors : fmt == QW_FMT_NF4_B64 ? 2 : 3;
  constexpr double kRound[4] = {2.1e-3, 2.4e-3, 2.3e-3, 2.4e-3};
  const double macs = (double)((M + 31) / 32 * 32) * N * K;
  const bool two = shape / 100 % 100 == 2 && K < 8192;  // 16-column blocks of a wave
  return 8 + fmax(K * kRound[f], macs / (f == 1 ? (two ? 45e6 : 75e6) : two ? 80e6 : 100e6));
}

// gemv: the call is one that a decode GEMV takes (fp16 activations, not gated).
Plan make_plan(const qw_weight &w, int M, bool gated, int x_dtype, bool gemv) {
  const int fmt = w.format, N = w.N, K = w.K, out_n = gated ? N / 2 : N;
  Plan p{Kernel::kNarrow, 0, 0, 1, false};
  const int forced = tune(QW_TUNE_LINEAR_ROW_BLOCKS);
  // Rows that a decode GEMV takes, if it can keep K whole (else its sums would go
  // through memory; up to four rows take the narrow kernel then). GEMV / narrow, us:
  //   2-bit, anchors   5120 x 5120, 1..3 rows   7.6/10.5  9.5/10.8  11.7/11.1
  //                   27648 x 5120            15.0/25.4 19.4/26.6  24.0/27.4
  //   2-bit            5120 x 5120             6.3/7.8   8.5/8.4   10.4/8.9
  //                    8192 x 8192             8.7/12.3 12.1/13.0  15.0/13.3
  //   NF4, 1 row 5120 x 5120 6.8/9.4;  INT4, anchors 8.5/10.4
  const int most_gemv = fmt == QW_FMT_2BIT_G32 ? (w.n_out > 0 ? 3 : 2) : 1;
  const int cols = tall_columns(gated), nt = (out_n + cols - 1) / cols;
  if (gemv && M <= most_gemv && forced <= 0) p.kernel = Kernel::kGemv;
  const int MR = forced > 0 && forced < 8 ? (forced == 4 ? 0 : forced) : M <= 4 ? 0 : M <= 16 ? 1 : 2;
  p.shape = pick_narrow(MR, fmt, out_n, K, gated);
  if (forced >= 8) {
    p.kernel = Kernel::kTall;
    p.high_tiles = forced >= 16 ? nt : 0;
  } else if (forced <= 0 && M > 32) {
    double least = narrow_time(fmt, w.n_out > 0, M, N, K, p.shape);
    auto consider = [&](double t, int high_tiles, int parts) {
      if (t >= least) return;
      least = t;
      p.kernel = Kernel::kTall;
      p.high_tiles = high_tiles;
      p.parts = parts;
    };
    for (int parts = 1; parts <= 16 && (parts == 1 || K / 64 / parts >= 2); parts *= 2) {
      consider(tall_time(fmt, w.n_out > 0, M, nt, N, K, false, parts), 0, parts);
      consider(tall_time(fmt, w.n_out > 0, M, nt, N, K, true, parts), nt, parts);
    }
    if (p.kernel == Kernel::kTall && p.parts == 1) p.high_tiles = pick_high_tiles(M, nt);
  }
  const int parts = tune(QW_TUNE_LINEAR_PARTS), step = p.kernel == Kernel::kTall ? 64 : 256;
  if (parts > 0) p.parts = parts < K / step ? parts : K / step > 1 ? K / step : 1;
  p.to_fp16 = p.kernel == Kernel::kTall && gated && x_dtype == QW_DT_BF16;
  return p;
}

// The rows of a tile lie within 32-bit offsets.
constexpr int kMostK = 1 << 22;

bool takes(const qw_weight *w, int M) {
  if (!w || M < 1 || M > QW_MAX_ROWS) return false;
  if (w->format != QW_FMT_2BIT_G32 && w->format != QW_FMT_NF4_B64 && w->format != QW_FMT_INT4_G32) return false;
  return w->N > 0 && w->K > 0 && w->K % 64 == 0 && w->K < kMostK && (unsigned long long)w->N * w->K < (1ull << 32);
}

template <int FMT>
qw_status run(const LinearArgs &a, const Plan &p, hipStream_t s) {
  if (p.kernel == Kernel::kTall) return launch_linear_tall<FMT>(a, p.high_tiles, s);
  return launch_linear_narrow<FMT>(a, p.shape, s);
}

}  // namespace
}  // namespace qw

extern "C" {

size_t qw_linear_workspace_bytes(const qw_weight *w, qw_dtype x_dtype, int M, int gated) {
  if (!qw::takes(w, M) || (gated && w->N % 2)) return 0;
  return qw::workspace_of(qw::make_plan(*w, M, gated != 0, x_dtype, false), M, w->N, w->K);
}

qw_status qgemm_linear(const qw_weight *w, const void *X, qw_dtype x_dtype, const float *x_scales, int M,
                       const qw_epilogue *ep, void *Y, qw_dtype y_dtype, void *workspace, size_t workspace_bytes,
                       void *stream) {
  using namespace qw;
  CallScope scope;
  if (!w || !X || !Y || M < 1 || !is_dtype(y_dtype)) return QW_ERR_INVALID_ARG;
  const bool in8 = x_dtype == QW_DT_E4M3 || x_dtype == QW_DT_I8;
  if (!in8 && x_dtype != QW_DT_F16 && x_dtype != QW_DT_BF16) return QW_ERR_INVALID_ARG;
  if (in8 != (x_scales != nullptr)) return QW_ERR_INVALID_ARG;
  if (w->format != QW_FMT_2BIT_G32 && w->format != QW_FMT_NF4_B64 && w->format != QW_FMT_INT4_G32)
    return QW_ERR_INVALID_ARG;
  QW_TRY(check_weight_view(w, w->format, 0));
  const qw_epilogue none{};
  if (!ep) ep = &none;
  if (ep->act < QW_ACT_NONE || ep->act > QW_ACT_GELU_TANH) return QW_ERR_INVALID_ARG;
  if ((ep->bias && !is_dtype(ep->bias_dtype)) || (ep->residual && !is_dtype(ep->residual_dtype))) return QW_ERR_INVALID_ARG;
  if (ep->gated && w->N % 2) return QW_ERR_INVALID_ARG;
  if (ep->residual == Y && ep->residual_dtype != y_dtype) return QW_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(x_scales) || !aligned16(Y) || !aligned16(ep->bias) || !aligned16(ep->residual))
    return QW_ERR_ALIGNMENT;
  if (!takes(w, M)) return QW_ERR_UNSUPPORTED;
  const size_t need = qw_linear_workspace_bytes(w, x_dtype, M, ep->gated);
  if (need && (!workspace || workspace_bytes < need)) return QW_ERR_INVALID_ARG;
  if (need && !aligned16(workspace)) return QW_ERR_ALIGNMENT;
  int cus = 0;
  QW_TRY(current_device(&cus));
  Plan plan = make_plan(*w, M, ep->gated != 0, x_dtype, x_dtype == QW_DT_F16 && !ep->gated);
  LinearArgs a{};
  a.X = X;
  a.codes = w->codes;
  a.scales = reinterpret_cast<const uint8_t *>(w->scales);
  a.idx = w->out_idx;
  a.mask = w->out_mask;
  a.wo = w->out_w;
  a.x_dtype = x_dtype;
  a.M = M;
  a.N = w->N;
  a.K = w->K;
  a.n_out = w->format == QW_FMT_NF4_B64 ? 0 : w->n_out;
  a.n_out_pad = w->n_out_pad;
  a.parts = plan.parts;
  const bool gated = ep->gated != 0;
  a.fin = Finish{x_scales, ep->bias, ep->residual, Y, reinterpret_cast<float *>(workspace), ep->bias_dtype, ep->residual_dtype,
                 (int)y_dtype, ep->act, gated, M, w->N, gated ? w->N / 2 : w->N};
  const float *L = nf4_levels_host();
  for (int i = 0; i < 16; ++i) a.nf4[i] = L[i];
  const hipStream_t s = as_stream(stream);
  if (plan.kernel == Kernel::kGemv) {
    const uint16_t *x = reinterpret_cast<const uint16_t *>(X);
    const qw_status st = w->format == QW_FMT_NF4_B64 ? launch_linear_gemv_nf4(*w, x, a.fin, cus, s)
                                                     : gemv2m::launch_linear(*w, x, M, a.fin, cus, s);
    if (st != QW_ERR_UNSUPPORTED) return st;
    plan = make_plan(*w, M, gated, x_dtype, false);
  }
  if (plan.to_fp16) {
    char *const at = reinterpret_cast<char *>(workspace) + parts_bytes(plan, M, w->N);
    float *const scales = reinterpret_cast<float *>(at + fp16_bytes(M, w->K));
    const int most = (int)kMostBlocks;
    for (int m = 0; m < M; m += most) {
      const int now = M - m < most ? M - m : most;
      QW_HIP_TRY(launch(to_fp16_kernel, (unsigned)now, 256, 0, s, reinterpret_cast<const uint16_t *>(X), reinterpret_cast<uint16_t *>(at),
                        scales, m, w->K));
    }
    a.X = at;
    a.x_dtype = QW_DT_F16;
    a.fin.x_scales = scales;
  }
  if (w->format == QW_FMT_2BIT_G32)
    QW_TRY(run<QW_FMT_2BIT_G32>(a, plan, s));
  else if (w->format == QW_FMT_INT4_G32)
    QW_TRY(run<QW_FMT_INT4_G32>(a, plan, s));
  else
    QW_TRY(run<QW_FMT_NF4_B64>(a, plan, s));
  if (plan.parts == 1) return QW_OK;
  const int col_blocks = (a.fin.out_n + 1023) / 1024;
  const int most = (int)(kMostBlocks / col_blocks);
  for (int m = 0; m < M; m += most) {
    const int now = M - m < most ? M - m : most;
    QW_HIP_TRY(launch(join_kernel, (unsigned)(now * col_blocks), 256, 0, s, a.fin, plan.parts, col_blocks, m));
  }
  return QW_OK;
}

}  // extern "C"
