// w4.h -- what the kernels of the 4-bit products share: the weights' decoding, the activation, the store.
//
// The matrix instructions take rows of x as their first operand and 16 outputs as their second; lane l
// holds row (output) l % 16, inputs of its quarter g = l / 16, and of the result column l % 16 (an
// output), rows 4 g + 0..3.
//
// INT codes enter the product as 16 + (code + 8) = code + 24, a shift and an and-or per pair: the four
// bits lie right below the exponent of 16.  Their product with a group of inputs starts from
// -24 sum(x), which the matrix cores form as one more product with a constant, shared by all outputs;
// the group's sum, exact products in 32 bits, is multiplied by its scale in 32 bits.  So no weight is
// rounded; what the detour adds is the rounding of 32-bit sums of up to 31 |x| instead of 8 |x|.
// MX codes are converted with their scale (a power of two: exact in BF16, whose exponents reach as far).
// F16 rows take them relative to the largest scale of the output, times 2^13 (the largest is then 6 2^13):
// exact down to 2^-36 of that scale, below it off by at most 2^-38 of it; the sum is scaled back once.
#pragma once

#include "layers.h"

namespace psispec {
namespace w4 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

struct F8 {};  // rows of e4m3 with a power of two per 32 inputs

__device__ inline f32x4 mfma(u32x4 x, u32x4 w, f32x4 c, __bf16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x),
                                                 __builtin_bit_cast(bf16x8, w), c, 0, 0, 0);
}
__device__ inline f32x4 mfma(u32x4 x, u32x4 w, f32x4 c, _Float16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x),
                                                __builtin_bit_cast(f16x8, w), c, 0, 0, 0);
}

// 8 INT codes (word of the packed layout) as code + 24
__device__ inline u32x4 int_codes(uint32_t w, __bf16) {
  return u32x4{((w << 3) & 0x00780078u) | 0x41804180u, ((w >> 1) & 0x00780078u) | 0x41804180u,
               ((w >> 5) & 0x00780078u) | 0x41804180u, ((w >> 9) & 0x00780078u) | 0x41804180u};
}
__device__ inline u32x4 int_codes(uint32_t w, _Float16) {
  return u32x4{((w << 6) & 0x03c003c0u) | 0x4c004c00u, ((w << 2) & 0x03c003c0u) | 0x4c004c00u,
               ((w >> 2) & 0x03c003c0u) | 0x4c004c00u, ((w >> 6) & 0x03c003c0u) | 0x4c004c00u};
}
// eight times -24
__device__ inline u32x4 minus24(__bf16) { return u32x4{0xc1c0c1c0u, 0xc1c0c1c0u, 0xc1c0c1c0u, 0xc1c0c1c0u}; }
__device__ inline u32x4 minus24(_Float16) { return u32x4{0xce00ce00u, 0xce00ce00u, 0xce00ce00u, 0xce00ce00u}; }

// 8 MX codes times the power of two whose exponent field `scale` holds
__device__ inline u32x4 mx_codes(uint32_t w, float scale, __bf16) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
}
__device__ inline u32x4 mx_codes(uint32_t w, float scale, _Float16) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3))};
}
// The scale under which a block's codes enter: byte e of the block, byte `top` of the output
__device__ inline float mx_scale(int e, int top, __bf16) { return __uint_as_float((uint32_t)e << 23); }
__device__ inline float mx_scale(int e, int top, _Float16) {
  return __uint_as_float((uint32_t)max(e - top + 140, 0) << 23);
}
// what the sum is multiplied by in the end
__device__ inline float mx_back(float acc, int top, __bf16) { return acc; }
__device__ inline float mx_back(float acc, int top, _Float16) {
  return top == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(acc, top - 140);
}

__device__ inline float scale16(uint32_t bits, bool f16) {
  return f16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)bits) : bf16_bits_to_f32((uint16_t)bits);
}

// 8 numbers of 8 bits times their power of two: exact in BF16 (values under 2^-126 lose bits, as its
// smallest numbers do)
__device__ inline u32x4 f8_rows(uint32_t lo, uint32_t hi, float scale) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true))};
}

__device__ inline float activate(float x, int act) {
  if (act == PSISPEC_W4_SILU) return x / (1.0f + expf(-x));
  if (act == PSISPEC_W4_GELU) return 0.5f * x * (1.0f + erff(x * 0.70710678118654752440f));
  const float u = 0.79788456080286535588f * (x + 0.044715f * x * x * x);  // sqrt(2 / pi) (x + ...)
  return 0.5f * x * (1.0f + tanhf(u));
}

__device__ inline float load16(const void* p, int64_t i, bool f16) {
  return scale16(static_cast<const uint16_t*>(p)[i], f16);
}
__device__ inline uint16_t round16(float v, bool f16) {
  return f16 ? __builtin_bit_cast(uint16_t, (_Float16)v) : __builtin_bit_cast(uint16_t, (__bf16)v);
}

// bias and rounding of a linear layer, or activation and product of a gated one
template <int MATS>
__device__ inline void store(const W4Args& a, int row, int n, float first, float second) {
  float y;
  if (MATS == 2)
    y = activate(first, a.act) * second;
  else
    y = a.bias ? first + load16(a.bias, n, a.out_f16) : first;
  static_cast<uint16_t*>(a.out)[(int64_t)row * a.out_stride + n] = round16(y, a.out_f16);
}

}  // namespace w4
}  // namespace psispec
