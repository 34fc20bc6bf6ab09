// w4.h -- what the kernels of the 4-bit products share: the weights' decoding, the activation, the store.
//
// The matrix instructions take 16 outputs as their first operand and 16 rows of x as their second; lane l
// holds output (row) l % 16, inputs of its quarter g = l / 16, and of the result outputs 4 g + 0..3 of row
// l % 16: neighbours, stored together.
//
// INT codes enter the product as 16 + (code + 8) = code + 24, a shift and an and-or per pair (the first
// needs no shift: 64 rows, 12288 x 4096 15.2 -> 14.5 us, 8000 rows 706 -> 696): the four
// bits lie right below the exponent of 16.  Their product with a group of inputs starts from
// -24 sum(x), which the matrix cores form as one more product with a constant, shared by all outputs;
// the group's sum, exact products in 32 bits, is multiplied by its scale in 32 bits.  So no weight is
// rounded; what the detour adds is the rounding of 32-bit sums of up to 31 |x| instead of 8 |x|.
// MX codes are converted with their scale (a power of two: exact in BF16, whose exponents reach as far but for the
// largest codes times 2^126 or 2^127: an output with such a scale takes all of its own one or two powers lower, the
// lowest as they are, and its sum is scaled back).
// F16 rows take them relative to the largest scale of the output, times 2^13 (the largest is then 6 2^13):
// exact down to 2^-36 of that scale, below it off by at most 2^-38 of it; the sum is scaled back once.
#pragma once

#include "layers.h"

namespace psispec {
namespace w4 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef uint64_t u64_any __attribute__((aligned(1)));

struct F8 {};  // rows of e4m3 with a power of two per 32 inputs

constexpr int kStageRow = 256;      // bytes of a row per step
constexpr int kRsrc3 = 0x00020000;  // raw buffer: reads out of range give 0
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) uint32_t global_u32;

// s_waitcnt: at most n loads in flight, the other counters as they are
constexpr int waitcnt_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }

// An LDS read.  The restrict-qualified parameter of an inlined function gives it an alias scope of its own, so
// that the compiler does not wait before it for every load to LDS in flight: the kernels order those and the
// reads themselves.
template <typename V>
__device__ __attribute__((always_inline)) inline V lds_read(const V* __restrict__ p) {
  return *p;
}

__device__ inline f32x4 mfma(u32x4 w, u32x4 x, f32x4 c, __bf16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w),
                                                 __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
}
__device__ inline f32x4 mfma(u32x4 w, u32x4 x, f32x4 c, _Float16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w),
                                                __builtin_bit_cast(f16x8, x), c, 0, 0, 0);
}

// The numbers of int_codes in registers: an and-or takes one literal at most, and two of them make the compiler
// split it.
struct IntBits {
  uint32_t mask, magic;
};
template <typename X>
__device__ inline IntBits int_bits() {
  IntBits b{__is_same(X, __bf16) ? 0x00780078u : 0x03c003c0u, __is_same(X, __bf16) ? 0x41804180u : 0x4c004c00u};
  asm("" : "+s"(b.mask));
  asm("" : "+v"(b.magic));
  return b;
}
// 8 INT codes (word of the packed layout, in which the first pair lies where BF16 wants it) as code + 24
__device__ inline uint32_t turn(uint32_t w, int by) { return __builtin_amdgcn_alignbit(w, w, by); }
__device__ inline u32x4 int_codes(uint32_t w, IntBits k, __bf16) {
  return u32x4{(w & k.mask) | k.magic, ((w >> 4) & k.mask) | k.magic, ((w >> 8) & k.mask) | k.magic,
               (turn(w, 12) & k.mask) | k.magic};
}
__device__ inline u32x4 int_codes(uint32_t w, IntBits k, _Float16) {
  return u32x4{((w << 3) & k.mask) | k.magic, ((w >> 1) & k.mask) | k.magic, ((w >> 5) & k.mask) | k.magic,
               (turn(w, 9) & k.mask) | k.magic};
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
// The scale under which a block's codes enter: byte e of the block, the largest byte `top` of the output.
// BF16: 252 at most, so that 6 times it is a number; two saturating subtractions
__device__ inline uint32_t mx_over(int top) { return __builtin_elementwise_sub_sat((uint32_t)top, 252u); }
__device__ inline float mx_scale(int e, int top, __bf16) {
  return __uint_as_float(__builtin_elementwise_sub_sat((uint32_t)e, mx_over(top)) << 23);
}
__device__ inline float mx_scale(int e, int top, _Float16) {
  return __uint_as_float((uint32_t)max(e - top + 140, 0) << 23);
}
// what the sum is multiplied by in the end
__device__ inline float mx_back(float acc, int top, __bf16) {
  return top == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(acc, (int)mx_over(top));
}
__device__ inline float mx_back(float acc, int top, _Float16) {
  return top == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(acc, top - 140);
}
// the same for a BF16 lane's sums of outputs 4 g + 0..3; lane l holds the byte of output l % 16
__device__ inline void mx_back4(f32x4& acc, int top) {
  const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = mx_back(acc[i], __shfl(top, 4 * g + i, 64), __bf16());
}

__device__ inline float scale16(uint32_t bits, bool f16) {
  return f16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)bits) : bf16_bits_to_f32((uint16_t)bits);
}

// The scales of the eight blocks from `blk` on of a row of 8-bit numbers; those behind the last of `all` are 1
// (their values are read as zeros)
__device__ inline uint64_t row_scales(const uint8_t* row, int blk, int all) {
  if (blk + 8 <= all) return *reinterpret_cast<const u64_any*>(row + blk);
  uint64_t v = 0x7f7f7f7f7f7f7f7full;
  for (int i = 0; i < all - blk; ++i) v = (v & ~(0xffull << (8 * i))) | (uint64_t)row[blk + i] << (8 * i);
  return v;
}

// 128 inputs of 16 outputs with MX weights (lane: inputs 32 g + 0..31) and of 16 rows of 8 bits (lane: inputs
// 16 g + 0..15 in x0, 64 + 16 g + 0..15 in x1; byte 0 of xs the scale of inputs 32 g ..),
// byte WS of ws that of the output.  Twice the 16-bit instructions' rate; what it costs: among eight
// neighbouring inputs each product is cut toward zero to a multiple of 2^-13 of the largest power of two that the
// factors' exponents add up to (at most that of the largest product); eights are joined in 32 bits.  A sum of
// products cut so in 64 bits gives the kernels' outputs to the last bit.  Why it is taken all the same: the rows' own
// rounding to 3 bits of mantissa is 2^-4 of each value, the cut moves the sums of 4096 random inputs with a few large
// columns by 1.4e-5 of their norm, the rounding to BF16 by 1.7e-3 (with it and with exact products alike), and exact
// products, the same rows in BF16 through the 16-bit instruction, take 33 us instead of 23 (576 rows, 6144 x 4096) and
// 21.6 instead of 16.9 (64 rows, 2 x 12288 x 4096 gated).
template <int WS>
__device__ inline f32x4 mfma_mx(u32x4 w, int ws, u32x4 x0, u32x4 x1, int xs, f32x4 c) {
  const i32x8 a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i32x8 b = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 0, WS, ws, 0, xs);
}

// 1 + erf(z) = erfc(-z) and 1 + tanh(u) = 2 / (1 + exp(-2 u)): without the loss of digits on the negative side, and
// by exp(-|u|), which does not overflow where x exp(u) is still a number (u to -91)
__device__ inline float activate(float x, int act) {
  if (act == PSISPEC_W4_GELU) return 0.5f * x * erfcf(-0.70710678118654752440f * x);
  const float u = act == PSISPEC_W4_SILU ? x : 1.59576912160573071176f * (x + 0.044715f * x * x * x);  // 2 sqrt(2 / pi)
  const float t = expf(-fabsf(u));
  return (u < 0.0f ? x * t : x) / (1.0f + t);
}

// The scales of the lane's outputs 4 g + 0..3, four numbers of 16 bits
template <bool F16>
__device__ inline f32x4 scales_of(u32x2 w) {
  return f32x4{scale16(w[0] & 0xffffu, F16), scale16(w[0] >> 16, F16), scale16(w[1] & 0xffffu, F16),
               scale16(w[1] >> 16, F16)};
}

__device__ inline float load16(const void* p, int64_t i, bool f16) {
  return scale16(static_cast<const uint16_t*>(p)[i], f16);
}
__device__ inline uint32_t round16(float v, bool f16) {
  return f16 ? __builtin_bit_cast(uint16_t, (_Float16)v) : __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Outputs n .. n + 3 of a row: bias and rounding of a linear layer, or activation and product of a gated one.
template <int MATS>
__device__ inline void store4(const W4Args& a, int64_t row, int n, f32x4 first, f32x4 second) {
  uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.out_stride + n;
  uint32_t y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float v;
    if (MATS == 2)
      v = activate(first[e], a.act) * second[e];
    else
      v = a.bias && n + e < a.n ? first[e] + load16(a.bias, n + e, a.out_f16) : first[e];
    y[e] = round16(v, a.out_f16);
  }
  if (a.out_vec && n + 4 <= a.n) {
    *reinterpret_cast<u32x2*>(out) = u32x2{y[0] | y[1] << 16, y[2] | y[3] << 16};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.n) out[e] = (uint16_t)y[e];
  }
}

}  // namespace w4
}  // namespace psispec
