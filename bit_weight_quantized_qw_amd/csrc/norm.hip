// The root-mean-square norm before a projection, with the residual stream's
// addition and the output in the form that the products take:
//   h[m][k] = x[m][k] + residual[m][k]
//   y[m][k] = h[m][k] / sqrt(mean_k h[m][k]^2 + eps) * weight[k]
// in 16 or 32 bits, or in 8 bits with one scale a row, optionally in the
// channel order of the INT4 format.
//
// What bounds it: memory, every element read once and written once. So a row
// stays in registers between its sums and its output, held by as many waves
// as that takes, and all of a lane's loads are requested before the first is
// used. h is fp32 in registers: what is normalised is the unrounded sum.
//
// The row's sum of squares and (8 bits) the largest |h weight| come from one
// pass and one exchange: the scale of a row is the largest y over the largest
// number of the type, and y is h weight times one factor a row. With perm, LDS
// turns the row: h weight in fp32, or the 8-bit elements as they are.
//
// Measured: 8192 x 8192 in bf16 with the residual, y in bf16 96 us (5.6 TB/s; a
// copy of 1 GiB here 5.2), in e4m3 89, permuted 102 (each
// byte by a read of LDS of its own); 8192 x 1024 11.6 us (5.8 TB/s); 777 x 5120 with an fp32 residual 10.2 us, in
// a permuted order 11.8; one row of 5120 4.2 us. Rows that do not start on 16 bytes
// (K not a multiple of 8) go by single elements: 4096 x 5119 70 us, 2.4 TB/s.
#include <math.h>

#include <type_traits>

#include "op16.h"

namespace qw {
namespace {

struct NormArgs {
  const void *x, *residual, *weight;
  const int32_t *perm;
  void *h_out, *y;
  float *y_scales;
  float eps;
  int M, K;
  int first;  // the launch's first row
  int x_dtype, r_dtype, w_dtype, y_dtype;
};

// V elements as they lie in memory, S bytes each.
template <int S, int V>
struct Raw {
  uint32_t w[S * V >= 4 ? S * V / 4 : 1];
};

template <int S, int V>
__device__ inline void load_raw(Raw<S, V> &d, const void *p, size_t i) {
  const char *at = reinterpret_cast<const char *>(p) + i * S;
  if constexpr (S * V >= 16) {
#pragma unroll
    for (int q = 0; q < S * V / 16; ++q) {
      const u32x4 v = reinterpret_cast<const u32x4 *>(at)[q];
      d.w[4 * q] = v[0]; d.w[4 * q + 1] = v[1]; d.w[4 * q + 2] = v[2]; d.w[4 * q + 3] = v[3];
    }
  } else if constexpr (S * V == 4) {
    d.w[0] = *reinterpret_cast<const uint32_t *>(at);
  } else {
    d.w[0] = *reinterpret_cast<const uint16_t *>(at);
  }
}

// Their numbers (of eight, dt is asked for once).
template <int S, int V>
__device__ inline void raw_values(const Raw<S, V> &d, float (&v)[V], int dt) {
  if constexpr (S == 4) {
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] = __builtin_bit_cast(float, d.w[q]);
  } else if constexpr (V == 1) {
    // both, and one of them by a mask (4096 x 5119 70 us, with a branch for each 73)
    uint32_t f16 = dt == QW_DT_F16 ? ~0u : 0u;
    asm("" : "+v"(f16));
    v[0] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, Op<QW_DT_F16>::value(d.w[0] & 0xFFFFu)) & f16) |
                                         (__builtin_bit_cast(uint32_t, Op<QW_DT_BF16>::value(d.w[0] & 0xFFFFu)) & ~f16));
  } else if (dt == QW_DT_F16) {
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] = Op<QW_DT_F16>::value((d.w[q / 2] >> (16 * (q & 1))) & 0xFFFFu);
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] = Op<QW_DT_BF16>::value((d.w[q / 2] >> (16 * (q & 1))) & 0xFFFFu);
  }
}

template <int DT>
__device__ inline void store_eight(uint16_t *o, const float (&v)[8]) {
  u32x4 w;
#pragma unroll
  for (int q = 0; q < 4; ++q) w[q] = Op<DT>::bits(v[2 * q]) | (Op<DT>::bits(v[2 * q + 1]) << 16);
  *reinterpret_cast<u32x4 *>(o) = w;
}
// Stores V values at element i, rounded to dt.
template <int V>
__device__ inline void store_values(void *p, size_t i, const float (&v)[V], int dt) {
  if (dt == QW_DT_F32) {
    float *o = reinterpret_cast<float *>(p) + i;
    if constexpr (V == 8) {
      reinterpret_cast<f32x4 *>(o)[0] = f32x4{v[0], v[1], v[2], v[3]};
      reinterpret_cast<f32x4 *>(o)[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      o[0] = v[0];
    }
    return;
  }
  uint16_t *o = reinterpret_cast<uint16_t *>(p) + i;
  if constexpr (V == 1)
    o[0] = (uint16_t)out_bits(v[0], dt);
  else if (dt == QW_DT_F16)
    store_eight<QW_DT_F16>(o, v);
  else
    store_eight<QW_DT_BF16>(o, v);
}

// V values as bytes of an 8-bit type; they are within its range but for a rounding
// of the scale's inverse.
template <int V>
struct Bytes {
  uint32_t w[V == 8 ? 2 : 1];
};
template <int V>
__device__ inline Bytes<V> to_8bit(const float (&v)[V], int dt) {
  Bytes<V> b = {};
  if (dt == QW_DT_I8) {
#pragma unroll
    for (int q = 0; q < V; ++q) {
      const int n = (int)rintf(__builtin_amdgcn_fmed3f(v[q], -127.0f, 127.0f));
      b.w[q / 4] |= ((uint32_t)n & 0xFFu) << (8 * (q & 3));
    }
  } else {
    float c[V];
#pragma unroll
    for (int q = 0; q < V; ++q) c[q] = __builtin_amdgcn_fmed3f(v[q], -448.0f, 448.0f);
    if constexpr (V == 8) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        b.w[q] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * q], c[4 * q + 1], 0, false);
        b.w[q] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * q + 2], c[4 * q + 3], (int)b.w[q], true);
      }
    } else {
      b.w[0] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[0], 0.0f, 0, false);
    }
  }
  return b;
}
template <int V>
__device__ inline void store_bytes(void *p, size_t i, const Bytes<V> &b) {
  uint8_t *o = reinterpret_cast<uint8_t *>(p) + i;
  if constexpr (V == 8)
    *reinterpret_cast<u32x2 *>(o) = u32x2{b.w[0], b.w[1]};
  else
    o[0] = (uint8_t)b.w[0];
}

// The smallest scale of a row: its inverse is finite, and rows of zeros (or of
// less than 2^-100 of the type's range) give zeros.
constexpr float kLeastScale = 0x1p-100f;

// XS, RS: bytes of an element of x and of the residual (0: none); W: waves of
// a row; IT: runs of V elements that a lane holds, at most. V is 8, or 1
// where rows do not start on 16 bytes.
// IN8: y in 8 bits; PERM: in a permuted order.
template <int XS, int RS, int W, int IT, int V, bool IN8, bool PERM>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void norm_kernel(NormArgs a) {
  constexpr int kRows = W == 1 ? 4 : 1;  // rows of a workgroup
  constexpr int kLanes = 64 * W;         // lanes of a row
  // with perm, the row in its own order: h weight in fp32, or 8-bit elements
  extern __shared__ __attribute__((aligned(16))) float smem[];  // [kRows][K] of either
  __shared__ double sums[W];
  __shared__ double tops[W];
  const int row_of = W == 1 ? (int)threadIdx.x >> 6 : 0;
  const int m = a.first + (int)blockIdx.x * kRows + row_of;
  if (m >= a.M) return;  // W == 1: whole waves, and no barrier below
  const int at = W == 1 ? (int)threadIdx.x & 63 : (int)threadIdx.x;
  const int K = a.K;
  const size_t row = (size_t)m * K;

  Raw<XS, V> xv[IT];
  Raw<RS ? RS : 2, V> rv[RS ? IT : 1];
  Raw<2, V> gv[IT];  // a weight in 16 bits, asked for with the row
  const bool w32 = a.w_dtype == QW_DT_F32;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int k = (i * kLanes + at) * V;
    if (k < K) load_raw(xv[i], a.x, row + k);
    if constexpr (RS != 0)
      if (k < K) load_raw(rv[i], a.residual, row + k);
    if (k < K && !w32) load_raw(gv[i], a.weight, k);
  }
  // the weights of run i: in registers, or 32-bit ones read again
  auto weights = [&](int i, int k, float (&g)[V]) {
    if (w32) {
      Raw<4, V> r;
      load_raw(r, a.weight, k);
      raw_values(r, g, QW_DT_F32);
    } else {
      raw_values(gv[i], g, a.w_dtype);
    }
  };
  float h[IT][V];
  // 8 bits: squares and products in 64 bits, so that a row's scale is its formula's,
  // rounded once (a scale that is off by a step moves all of the row's elements
  // towards the next borders of the grid)
  std::conditional_t<IN8, double, float> part = 0;
  double top = 0.0;         // the largest |h weight|; infinite beside an infinity or a NaN
  double not_finite = 0.0;  // no number then
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int k = (i * kLanes + at) * V;
    if (k >= K) continue;
    raw_values(xv[i], h[i], a.x_dtype);
    if constexpr (RS != 0) {
      float r[V];
      raw_values(rv[i], r, a.r_dtype);
#pragma unroll
      for (int q = 0; q < V; ++q) h[i][q] += r[q];
    }
#pragma unroll
    for (int q = 0; q < V; ++q) {
      if constexpr (IN8)
        part = __builtin_fma((double)h[i][q], (double)h[i][q], part);
      else
        part = __builtin_fmaf(h[i][q], h[i][q], part);
    }
    if (RS != 0 && a.h_out) store_values<V>(a.h_out, row + k, h[i], a.r_dtype);
    float g[V];
    weights(i, k, g);
    if constexpr (IN8) {
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const double p = (double)h[i][q] * (double)g[q];
        top = fmax(top, fabs(p));
        not_finite += p;
      }
    } else if constexpr (PERM) {
#pragma unroll
      for (int q = 0; q < V; ++q) smem[(size_t)row_of * K + k + q] = h[i][q] * g[q];
    } else {
#pragma unroll
      for (int q = 0; q < V; ++q) h[i][q] *= g[q];
    }
  }
  // the lanes' sums are added, and the row's factors computed, in 64 bits
  double sum = (double)part;
  if (IN8 && !(fabs(not_finite) < (double)INFINITY)) top = (double)INFINITY;
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    sum += __shfl_xor(sum, d, 64);
    if constexpr (IN8) top = fmax(top, __shfl_xor(top, d, 64));
  }
  // the row's LDS is written before any of it is read
  auto row_written = [&]() {
    if constexpr (W > 1) {
      __syncthreads();
    } else {  // by one wave
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    }
  };
  if constexpr (W > 1) {
    const int wv = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      sums[wv] = sum;
      tops[wv] = top;
    }
    row_written();
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      sum += sums[w];
      if constexpr (IN8) top = fmax(top, tops[w]);
    }
  } else {
    row_written();
  }
  const double inv = 1.0 / sqrt(sum / (double)K + (double)a.eps);
  float f = (float)inv;
  float f_rest = 0.0f;  // what f's rounding left
  if constexpr (IN8) {
    const double most = a.y_dtype == QW_DT_I8 ? 127.0 : 448.0;
    const double largest = top * inv;
    // a row with an infinity or a NaN has no scale
    const bool fine = top <= (double)__FLT_MAX__ && largest < (double)INFINITY;
    const float scale = fine ? fmaxf((float)(largest / most), kLeastScale) : NAN;
    if (at == 0) a.y_scales[m] = scale;
    double factor = fine ? inv / (double)scale : 0.0;
    // tiny rows by tiny weights (eps as small, or the least scale): the factor may lie
    // past fp32's range, so h takes a part of it (h weight is below 2^-91 then)
    if (factor > 0x1p100) {
      factor *= 0x1p-64;
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int q = 0; q < V; ++q) h[i][q] *= 0x1p64f;
    }
    f = (float)factor;
    f_rest = (float)(factor - (double)f);
  }
  uint8_t *const bytes = reinterpret_cast<uint8_t *>(smem) + (size_t)row_of * K;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int k = (i * kLanes + at) * V;
    if (k >= K) continue;
    float v[V];
    if constexpr (IN8) {
      float g[V];
      weights(i, k, g);
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const float p = h[i][q] * g[q];
        // rounded once, so that only values next to a border of the grid could
        // fall on its other side; infinity times zero is not zero
        v[q] = f == 0.0f ? 0.0f : __builtin_fmaf(p, f, __builtin_fmaf(p, f_rest, __builtin_fmaf(h[i][q], g[q], -p) * f));
      }
      const Bytes<V> b = to_8bit<V>(v, a.y_dtype);
      if constexpr (PERM)
        store_bytes<V>(bytes, k, b);
      else
        store_bytes<V>(a.y, row + k, b);
    } else {
      if constexpr (PERM) {
        Raw<4, V> from;
        load_raw(from, a.perm, k);
#pragma unroll
        for (int q = 0; q < V; ++q) v[q] = from.w[q] < (uint32_t)K ? smem[(size_t)row_of * K + from.w[q]] * f : 0.0f;
      } else {
#pragma unroll
        for (int q = 0; q < V; ++q) v[q] = h[i][q] * f;
      }
      store_values<V>(a.y, row + k, v, a.y_dtype);
    }
  }
  if constexpr (IN8 && PERM) {  // elements take the other order as they are
    row_written();
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int k = (i * kLanes + at) * V;
      if (k >= K) continue;
      Raw<4, V> from;
      load_raw(from, a.perm, k);
      Bytes<V> b = {};
#pragma unroll
      for (int q = 0; q < V; ++q)
        if (from.w[q] < (uint32_t)K) b.w[q / 4] |= (uint32_t)bytes[from.w[q]] << (8 * (q & 3));
      store_bytes<V>(a.y, row + k, b);
    }
  }
}

template <int XS, int RS, int W, int IT, int V, bool IN8, bool PERM>
qw_status launch_form(NormArgs a, hipStream_t s) {
  constexpr auto kernel = norm_kernel<XS, RS, W, IT, V, IN8, PERM>;
  constexpr int kRows = W == 1 ? 4 : 1, kThreads = W == 1 ? 256 : 64 * W;
  const size_t lds = PERM ? (size_t)kRows * a.K * (IN8 ? 1 : sizeof(float)) : 0;
  if (lds > 32768)
    QW_HIP_TRY(hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds));
  constexpr int kMost = (int)(0xFFFFFFFFll / kThreads) * kRows;  // a launch counts its threads in 32 bits
  for (; a.first < a.M; a.first += kMost) {
    const int rows = a.M - a.first < kMost ? a.M - a.first : kMost;
    QW_HIP_TRY(launch(kernel, (unsigned)((rows + kRows - 1) / kRows), kThreads, lds, s, a));
  }
  return QW_OK;
}

template <int XS, int RS, int W, int IT, int V>
qw_status launch_one(const NormArgs &a, hipStream_t s) {
  if (a.y_dtype == QW_DT_E4M3 || a.y_dtype == QW_DT_I8)
    return a.perm ? launch_form<XS, RS, W, IT, V, true, true>(a, s) : launch_form<XS, RS, W, IT, V, true, false>(a, s);
  return a.perm ? launch_form<XS, RS, W, IT, V, false, true>(a, s) : launch_form<XS, RS, W, IT, V, false, false>(a, s);
}

template <int XS, int RS>
qw_status launch_sizes(const NormArgs &a, hipStream_t s) {
  const int K = a.K;
  if (K % 8 == 0) {
    if (K <= 512) return launch_one<XS, RS, 1, 1, 8>(a, s);
    if (K <= 2048) return launch_one<XS, RS, 1, 4, 8>(a, s);
    if (K <= 4096) return launch_one<XS, RS, 4, 2, 8>(a, s);
    if (K <= 8192) return launch_one<XS, RS, 4, 4, 8>(a, s);
    if (K <= 16384) return launch_one<XS, RS, 16, 2, 8>(a, s);
    return launch_one<XS, RS, 16, 4, 8>(a, s);
  }
  if (K <= 512) return launch_one<XS, RS, 1, 8, 1>(a, s);
  if (K <= 8192) return launch_one<XS, RS, 4, 32, 1>(a, s);
  return launch_one<XS, RS, 16, 32, 1>(a, s);
}

template <int XS>
qw_status launch_residual(const NormArgs &a, hipStream_t s) {
  if (!a.residual) return launch_sizes<XS, 0>(a, s);
  return a.r_dtype == QW_DT_F32 ? launch_sizes<XS, 4>(a, s) : launch_sizes<XS, 2>(a, s);
}

}  // namespace
}  // namespace qw

extern "C" qw_status qw_rmsnorm(const void *x, qw_dtype x_dtype, const void *residual, qw_dtype residual_dtype,
                                const void *weight, qw_dtype weight_dtype, float eps, int M, int K,
                                const int32_t *perm, void *residual_out, void *y, qw_dtype y_dtype,
                                float *y_scales, void *stream) {
  using namespace qw;
  CallScope scope;
  if (!x || !weight || !y || M < 1 || K < 1) return QW_ERR_INVALID_ARG;
  if (!is_dtype(x_dtype) || !is_dtype(weight_dtype)) return QW_ERR_INVALID_ARG;
  if (residual ? !is_dtype(residual_dtype) : residual_out != nullptr) return QW_ERR_INVALID_ARG;
  const bool in8 = y_dtype == QW_DT_E4M3 || y_dtype == QW_DT_I8;
  if (!in8 && !is_dtype(y_dtype)) return QW_ERR_INVALID_ARG;
  if (in8 != (y_scales != nullptr)) return QW_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !(eps < INFINITY)) return QW_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(perm) || !aligned16(residual_out) ||
      !aligned16(y) || !aligned16(y_scales))
    return QW_ERR_ALIGNMENT;
  if (K > QW_MAX_NORM_K || M > QW_MAX_ROWS) return QW_ERR_UNSUPPORTED;
  QW_TRY(current_device(nullptr));
  const NormArgs a{x, residual, weight, perm, residual_out, y, y_scales, eps, M, K, 0, x_dtype, residual_dtype, weight_dtype, y_dtype};
  return x_dtype == QW_DT_F32 ? launch_residual<4>(a, as_stream(stream)) : launch_residual<2>(a, as_stream(stream));
}
