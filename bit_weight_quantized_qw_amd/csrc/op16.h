// 16-bit operand types of the matrix cores (16 x 16 x 32 products, fp32 sums)
// and the conversions around them.
#pragma once

#include "qw_internal.h"

namespace qw {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A operand: lane l holds row l % 16, elements 8 (l / 16) .. + 7 of the 32;
// B operand: column l % 16, the same elements; result: column l % 16, rows
// 4 (l / 16) .. + 3.
template <int DT>
struct Op;
template <>
struct Op<QW_DT_F16> {
  typedef _Float16 frag __attribute__((ext_vector_type(8)));
  static __device__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c, 0, 0, 0);
  }
  static __device__ uint32_t bits(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
  static __device__ float value(uint32_t b) { return f16_bits_to_f32((uint16_t)b); }
};
template <>
struct Op<QW_DT_BF16> {
  typedef __bf16 frag __attribute__((ext_vector_type(8)));
  static __device__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c, 0, 0, 0);
  }
  static __device__ uint32_t bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
  static __device__ float value(uint32_t b) { return __builtin_bit_cast(float, b << 16); }
};

__device__ inline uint32_t out_bits(float v, int dt) {
  return dt == QW_DT_F16 ? Op<QW_DT_F16>::bits(v) : Op<QW_DT_BF16>::bits(v);
}

inline bool is_dtype(int d) { return d == QW_DT_F16 || d == QW_DT_BF16 || d == QW_DT_F32; }

}  // namespace qw
