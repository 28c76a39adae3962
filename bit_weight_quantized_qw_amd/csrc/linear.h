// What the kernels of qgemm_linear share: the arguments, the activations as
// they lie in memory, and what is applied to the fp32 sums.
#pragma once

#include "experts.h"

namespace qw {

// What stands behind the sums, and where it goes.
struct Finish {
  const float *x_scales;    // [M], null for 16-bit activations
  const void *bias, *residual;
  void *Y;                  // [M][out_n]
  float *partial;           // [parts][M][N] where K is cut into parts
  int bias_dtype, residual_dtype, y_dtype;
  int act, gated;
  int M, N, out_n;          // out_n: N, gated N / 2
};

struct LinearArgs {
  const void *X;            // [M][K]
  const uint8_t *codes;
  const uint8_t *scales;
  const int32_t *idx;       // 2-bit anchors [n_out]
  const uint32_t *mask;     // 2-bit anchors [K/32]
  const uint16_t *wo;       // anchors [N][n_out_pad], fp16
  int x_dtype;
  int M, N, K;
  int n_out, n_out_pad;
  int row_tiles, col_tiles, parts;
  Finish fin;
  float nf4[16];
};

// Element i of a vector of a 16- or 32-bit type.
__device__ inline float load_any(const void *p, size_t i, int dt) {
  if (dt == QW_DT_F32) return reinterpret_cast<const float *>(p)[i];
  const uint32_t b = reinterpret_cast<const uint16_t *>(p)[i];
  return dt == QW_DT_F16 ? Op<QW_DT_F16>::value(b) : Op<QW_DT_BF16>::value(b);
}
// Four 16-bit numbers.
__device__ inline f32x4 four_of(u32x2 w, int dt) {
  if (dt == QW_DT_F16)
    return f32x4{Op<QW_DT_F16>::value(w[0] & 0xFFFFu), Op<QW_DT_F16>::value(w[0] >> 16), Op<QW_DT_F16>::value(w[1] & 0xFFFFu),
                 Op<QW_DT_F16>::value(w[1] >> 16)};
  return f32x4{Op<QW_DT_BF16>::value(w[0] & 0xFFFFu), Op<QW_DT_BF16>::value(w[0] >> 16), Op<QW_DT_BF16>::value(w[1] & 0xFFFFu),
               Op<QW_DT_BF16>::value(w[1] >> 16)};
}
// Four of a vector from i on; vec: i is a multiple of four elements.
__device__ inline f32x4 load_four(const void *p, size_t i, int dt, int count, bool vec) {
  f32x4 v = {0, 0, 0, 0};
  if (vec && count >= 4) {
    if (dt == QW_DT_F32) return *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(p) + i);
    return four_of(*reinterpret_cast<const u32x2 *>(reinterpret_cast<const uint16_t *>(p) + i), dt);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (q < count) v[q] = load_any(p, i + q, dt);
  return v;
}

// The activation of four values; act is uniform.
__device__ inline f32x4 activate(f32x4 z, int act) {
  switch (act) {
    case QW_ACT_RELU:
#pragma unroll
      for (int q = 0; q < 4; ++q) z[q] = z[q] < 0.0f ? 0.0f : z[q];  // keeps a NaN
      break;
    case QW_ACT_SILU:
#pragma unroll
      for (int q = 0; q < 4; ++q) z[q] = z[q] / (1.0f + expf(-z[q]));
      break;
    case QW_ACT_GELU:
#pragma unroll
      for (int q = 0; q < 4; ++q) z[q] = 0.5f * z[q] * erfcf(-0.70710678118654752f * z[q]);
      break;
    case QW_ACT_GELU_TANH:
      // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)): no cancellation far below zero
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float u = 0.79788456080286536f * (z[q] + 0.044715f * z[q] * z[q] * z[q]);
        z[q] = z[q] / (1.0f + expf(-2.0f * u));
      }
      break;
  }
  return z;
}

// What stands behind four sums (up: those of the up columns where gated) but the
// residual: the row's scale, the columns' bias, the activation, the gate.
__device__ inline f32x4 shape_values(const Finish &a, f32x4 s, f32x4 up, float scale, f32x4 bias, f32x4 bias_up) {
#pragma unroll
  for (int q = 0; q < 4; ++q) s[q] = __builtin_fmaf(s[q], scale, bias[q]);
  s = activate(s, a.act);
  if (a.gated) {
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] *= __builtin_fmaf(up[q], scale, bias_up[q]);
  }
  return s;
}
// Stores four values at columns n.. of row m, those below out_n.
__device__ inline void store_four(const Finish &a, int m, int n, f32x4 s) {
  const size_t o = (size_t)m * a.out_n + n;
  if (a.out_n % 4 == 0 && n + 4 <= a.out_n) {
    if (a.y_dtype == QW_DT_F32)
      *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(a.Y) + o) = s;
    else
      *reinterpret_cast<u32x2 *>(reinterpret_cast<uint16_t *>(a.Y) + o) =
          u32x2{out_bits(s[0], a.y_dtype) | (out_bits(s[1], a.y_dtype) << 16),
                out_bits(s[2], a.y_dtype) | (out_bits(s[3], a.y_dtype) << 16)};
    return;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (n + q >= a.out_n) continue;
    if (a.y_dtype == QW_DT_F32)
      reinterpret_cast<float *>(a.Y)[o + q] = s[q];
    else
      reinterpret_cast<uint16_t *>(a.Y)[o + q] = (uint16_t)out_bits(s[q], a.y_dtype);
  }
}

// The inputs of four columns n.. of row m.
__device__ inline float scale_at(const Finish &a, int m) { return a.x_scales ? a.x_scales[m] : 1.0f; }
__device__ inline f32x4 bias_at(const Finish &a, int n) {
  return a.bias ? load_four(a.bias, n, a.bias_dtype, a.out_n - n, true) : f32x4{0, 0, 0, 0};
}
__device__ inline f32x4 bias_up_at(const Finish &a, int n) {
  return a.bias && a.gated ? load_four(a.bias, (size_t)a.out_n + n, a.bias_dtype, a.out_n - n, a.out_n % 4 == 0) : f32x4{0, 0, 0, 0};
}
__device__ inline f32x4 residual_at(const Finish &a, int m, int n) {
  return a.residual ? load_four(a.residual, (size_t)m * a.out_n + n, a.residual_dtype, a.out_n - n, a.out_n % 4 == 0) : f32x4{0, 0, 0, 0};
}

// All of it for one sum, column n of row m (not gated).
__device__ inline void finish_one(const Finish &a, int m, int n, float v, float bias, float residual) {
  v = activate(f32x4{v * scale_at(a, m) + bias, 0, 0, 0}, a.act)[0] + residual;
  const size_t o = (size_t)m * a.out_n + n;
  if (a.y_dtype == QW_DT_F32)
    reinterpret_cast<float *>(a.Y)[o] = v;
  else
    reinterpret_cast<uint16_t *>(a.Y)[o] = (uint16_t)out_bits(v, a.y_dtype);
}
__device__ inline void finish_one(const Finish &a, int m, int n, float v) {
  finish_one(a, m, n, v, a.bias ? load_any(a.bias, n, a.bias_dtype) : 0.0f,
             a.residual ? load_any(a.residual, (size_t)m * a.out_n + n, a.residual_dtype) : 0.0f);
}

// Four sums of a part of K: columns n.. of row m, those below `end`.
__device__ inline void store_part(const Finish &a, int part, int m, int n, int end, f32x4 v) {
  float *const o = a.partial + ((size_t)part * a.M + m) * a.N + n;
  if (n + 4 <= end && a.out_n % 4 == 0) {  // then N is a multiple of 4, and n always
    *reinterpret_cast<f32x4 *>(o) = v;
    return;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (n + q < end) o[q] = v[q];
}

// Activations as operands of type DT (the matrix cores' 16-bit types): eight
// consecutive elements as loaded, and as the operand. 8-bit types become fp16
// exactly: e4m3 has 4 significant bits and 2^-9 .. 448, int8 8 bits (its bytes,
// plus 128, are put behind the exponent of 1024).
template <int XT>
struct XLoad {
  static constexpr bool k8 = XT == QW_DT_E4M3 || XT == QW_DT_I8;
  static constexpr int kBytes = k8 ? 1 : 2;
  static constexpr int DT = XT == QW_DT_BF16 ? QW_DT_BF16 : QW_DT_F16;
  typedef uint32_t raw __attribute__((ext_vector_type(k8 ? 2 : 4)));
  // at byte `offset` (a lane's, kOob reads zeros) + `scalar` (uniform)
  static __device__ raw load(__amdgpu_buffer_rsrc_t r, uint32_t offset, int scalar) {
    if constexpr (k8)
      return __builtin_amdgcn_raw_buffer_load_b64(r, (int)offset, scalar, 0);
    else
      return __builtin_amdgcn_raw_buffer_load_b128(r, (int)offset, scalar, 0);
  }
  static __device__ u32x4 operand(raw r) {
    if constexpr (XT == QW_DT_E4M3) {
      const uint32_t a = r[0], b = r[1];
      return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true))};
    } else if constexpr (XT == QW_DT_I8) {
      typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
      const f16x2 off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
      u32x4 o;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t w = r[q >> 1], u = w ^ 0x80808080u;
        const f16x2 v = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, q & 1 ? 0x04030402u : 0x04010400u)) + off;
        o[q] = __builtin_bit_cast(uint32_t, v);
      }
      return o;
    } else {
      return r;
    }
  }
};

// One element of activations, as 16 bits of DT.
template <int XT, int DT>
__device__ inline uint32_t one_as_16(const void *p, size_t element) {
  static_assert(DT == XLoad<XT>::DT, "the operands' type");
  if constexpr (XT == QW_DT_I8) {
    return Op<DT>::bits((float)reinterpret_cast<const int8_t *>(p)[element]);
  } else if constexpr (XT == QW_DT_E4M3) {
    const uint32_t b = reinterpret_cast<const uint8_t *>(p)[element];
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false)) & 0xFFFFu;
  } else {
    return reinterpret_cast<const uint16_t *>(p)[element];
  }
}

// The decode GEMVs with what stands behind the sums in their epilogue, fp16
// activations, not gated: 2-bit up to three rows and INT4 one row on the matrix
// cores (gemv2_mfma.hip), NF4 one row (gemv_nf4.hip). QW_ERR_UNSUPPORTED
// (nothing enqueued) where the shape does not fit them in one pass.
namespace gemv2m {
qw_status launch_linear(const qw_weight &w, const uint16_t *x, int M, const Finish &fin, int cus, hipStream_t s);
}
qw_status launch_linear_gemv_nf4(const qw_weight &w, const uint16_t *x, const Finish &fin, int cus, hipStream_t s);

// The narrow kernel of one format (linear_narrow_*.hip): tiles of 16 MR rows (MR
// = 0: of four) times 16 SUB columns by W waves.
constexpr int narrow_shape(int MR, int SUB, int W) { return MR * 10000 + SUB * 100 + W; }
template <int FMT>
qw_status launch_linear_narrow(const LinearArgs &a, int shape, hipStream_t s);
// The tall kernel of one format (linear_tall_*.hip): the first high_tiles tiles
// of columns by 256 rows, the others by 128.
constexpr int tall_columns(bool gated) { return gated ? 128 : 256; }  // columns of Y of a tile
template <int FMT>
qw_status launch_linear_tall(const LinearArgs &a, int high_tiles, hipStream_t s);

}  // namespace qw
