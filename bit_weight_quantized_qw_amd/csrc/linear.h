// What the kernels of qgemm_linear share: the arguments, the activations as
// they lie in memory, and what is applied to the fp32 sums.
#pragma once

#include "experts.h"

namespace qw {

struct LinearArgs {
  const void *X;            // [M][K]
  const float *x_scales;    // [M], null for 16-bit activations
  const uint8_t *codes;
  const uint8_t *scales;
  const int32_t *idx;       // 2-bit anchors [n_out]
  const uint32_t *mask;     // 2-bit anchors [K/32]
  const uint16_t *wo;       // anchors [N][n_out_pad], fp16
  void *Y;                  // [M][out_n]
  float *partial;           // [parts][M][N] where K is cut into parts
  const void *bias, *residual;
  int bias_dtype, residual_dtype, act, gated;
  int x_dtype, y_dtype;
  int M, N, K, out_n;
  int n_out, n_out_pad;
  int row_tiles, col_tiles, parts;
  float nf4[16];
};

// Element i of a vector of a 16- or 32-bit type.
__device__ inline float load_any(const void *p, size_t i, int dt) {
  if (dt == QW_DT_F32) return reinterpret_cast<const float *>(p)[i];
  const uint32_t b = reinterpret_cast<const uint16_t *>(p)[i];
  return dt == QW_DT_F16 ? Op<QW_DT_F16>::value(b) : Op<QW_DT_BF16>::value(b);
}
// Four of them from i on; vec: i is a multiple of four elements.
__device__ inline f32x4 load_four(const void *p, size_t i, int dt, int count, bool vec) {
  f32x4 v = {0, 0, 0, 0};
  if (vec && count >= 4) {
    if (dt == QW_DT_F32) return *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(p) + i);
    const u32x2 w = *reinterpret_cast<const u32x2 *>(reinterpret_cast<const uint16_t *>(p) + i);
    if (dt == QW_DT_F16)
      return f32x4{Op<QW_DT_F16>::value(w[0] & 0xFFFFu), Op<QW_DT_F16>::value(w[0] >> 16), Op<QW_DT_F16>::value(w[1] & 0xFFFFu),
                   Op<QW_DT_F16>::value(w[1] >> 16)};
    return f32x4{Op<QW_DT_BF16>::value(w[0] & 0xFFFFu), Op<QW_DT_BF16>::value(w[0] >> 16), Op<QW_DT_BF16>::value(w[1] & 0xFFFFu),
                 Op<QW_DT_BF16>::value(w[1] >> 16)};
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (q < count) v[q] = load_any(p, i + q, dt);
  return v;
}

// The activation; act is uniform.
__device__ inline float activate(float z, int act) {
  switch (act) {
    case QW_ACT_RELU: return z < 0.0f ? 0.0f : z;  // keeps a NaN
    case QW_ACT_SILU: return z / (1.0f + expf(-z));
    case QW_ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    case QW_ACT_GELU_TANH: {
      // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)): no cancellation far below zero
      const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
      return z / (1.0f + expf(-2.0f * u));
    }
  }
  return z;
}

// What stands behind the sums of four columns n.. of row m: s the sums, up the
// sums of the up columns where gated. Stores the columns below out_n.
__device__ inline void finish_four(const LinearArgs &a, int m, int n, f32x4 s, f32x4 up) {
  const int count = a.out_n - n;
  const bool vec = a.out_n % 4 == 0;
  if (a.x_scales) {
    const float f = a.x_scales[m];
    s *= f;
    if (a.gated) up *= f;
  }
  if (a.bias) {
    s += load_four(a.bias, n, a.bias_dtype, count, true);
    if (a.gated) up += load_four(a.bias, (size_t)a.out_n + n, a.bias_dtype, count, vec);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) s[q] = activate(s[q], a.act);
  if (a.gated) s *= up;
  const size_t o = (size_t)m * a.out_n + n;
  if (a.residual) s += load_four(a.residual, o, a.residual_dtype, count, vec);
  if (vec && count >= 4) {
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
    if (q >= count) continue;
    if (a.y_dtype == QW_DT_F32)
      reinterpret_cast<float *>(a.Y)[o + q] = s[q];
    else
      reinterpret_cast<uint16_t *>(a.Y)[o + q] = (uint16_t)out_bits(s[q], a.y_dtype);
  }
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
  static __device__ raw load(const void *p, size_t element) {
    return *reinterpret_cast<const raw *>(reinterpret_cast<const char *>(p) + element * kBytes);
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
  // one element, as 16 bits of DT
  static __device__ uint32_t one(const void *p, size_t element) {
    if constexpr (XT == QW_DT_I8) {
      return Op<QW_DT_F16>::bits((float)reinterpret_cast<const int8_t *>(p)[element]);
    } else if constexpr (XT == QW_DT_E4M3) {
      const uint32_t b = reinterpret_cast<const uint8_t *>(p)[element];
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false)) & 0xFFFFu;
    } else {
      return reinterpret_cast<const uint16_t *>(p)[element];
    }
  }
};

}  // namespace qw
