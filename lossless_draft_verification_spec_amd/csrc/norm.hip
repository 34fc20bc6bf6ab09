// norm.hip -- the residual's addition and the root-mean-square norm, in one pass over the rows.
//
//   h = x + residual;  residual_out = h;  y = h / sqrt(mean(h^2) + eps) * weight
//   8 bits: q = y / s, s = max|y| / 448 per row, or per 32 columns the smallest power of two with
//   max|y| <= 448 s
//
// A row stays in the registers of its threads between the sum of squares and the output, so every
// element is read once and written once.  A thread holds chunks of 8 elements, TPR chunks apart: a
// wave reads 1 KB at a time, and the 32 columns of a power-of-two scale belong to four neighbouring
// lanes.  h is squared and normalised as the 32-bit sum, before residual_out rounds it.  BF16 and 32-bit
// rows reach numbers whose squares 32 bits do not hold: such a row is summed again in 64 bits (all rows in
// 64 bits: 2% more for 8000 rows of 5120).
// Bound by memory: 8000 rows of 5120 (F16, residual in 32 bits, out in 8 bits) 84 us, 5.4 TB/s, where a large copy
// reaches 5.1; 576 rows of 4096 6 us and one row 3.5, the launch and one round of loads.
#include "layers.h"

namespace psispec {
namespace {

// Rows may start anywhere: vectors of their elements' alignment, which global memory takes as they are (8000 rows of
// 4096 with a residual, every second one off 16 bytes: 62 us, element by element 149; all of them on 16 bytes 55)
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8), aligned(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2), aligned(1)));
template <typename T> struct Vec8;
template <> struct Vec8<__bf16> { typedef bf16x8 type; };
template <> struct Vec8<_Float16> { typedef f16x8 type; };

// 8 elements of a row from column c on; those from dim on are 0.
template <typename T>
__device__ inline void load8(const T* row, int c, int dim, float* v) {
  if (c + 8 <= dim) {
    if constexpr (sizeof(T) == 4) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(row + c), b = *reinterpret_cast<const f32x4*>(row + c + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
    } else {
      const typename Vec8<T>::type a = *reinterpret_cast<const typename Vec8<T>::type*>(row + c);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (float)a[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < dim ? (float)row[c + e] : 0.0f;
  }
}

template <typename T>
__device__ inline void store8(T* row, int c, int dim, const float* v) {
  if (c + 8 <= dim) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<f32x4*>(row + c) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(row + c + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      typename Vec8<T>::type a;
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = (T)v[e];
      *reinterpret_cast<typename Vec8<T>::type*>(row + c) = a;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < dim) row[c + e] = (T)v[e];
  }
}

// 8 values, clamped to +-448 (NaN stays) and rounded to nearest
__device__ inline u32x2 pack8_e4m3(const float* v) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = v[e] == v[e] ? fminf(fmaxf(v[e], -448.0f), 448.0f) : v[e];
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int u = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], u, true);
  }
  return w;
}

// Reductions over the threads of a row: within the wave, then over its waves in a fixed order.
template <int TPR, typename S>
__device__ inline S row_sum(S v, S* lds) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (TPR == 64) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  S s = 0;
#pragma unroll
  for (int w = 0; w < TPR / 64; ++w) s += lds[w];
  return s;
}
template <int TPR>
__device__ inline uint32_t row_max(uint32_t v, uint32_t* lds) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  if constexpr (TPR == 64) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < TPR / 64; ++w) m = max(m, lds[w]);
  return m;
}

// T: x, weight and 16-bit out; R: residual; KIND: NormOut; TPR threads per row, each with up to CPT
// chunks of 8.
template <typename T, typename R, int KIND, int TPR, int CPT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_add_rmsnorm(AddNormArgs a) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
  __shared__ float s_sum[TPR / 64];
  __shared__ double s_wide[TPR / 64];
  __shared__ uint32_t s_max[TPR / 64];
  const int u = kRows > 1 ? (int)threadIdx.x % TPR : (int)threadIdx.x;
  const int64_t row = (int64_t)blockIdx.x * kRows + (kRows > 1 ? (int)threadIdx.x / TPR : 0);
  if (kRows > 1 && row >= a.rows) return;  // whole waves, and no barrier with 64 threads per row
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const R* res = a.residual ? static_cast<const R*>(a.residual) + row * a.residual_stride : nullptr;
  R* ro = a.residual_out ? static_cast<R*>(a.residual_out) + row * a.residual_out_stride : nullptr;
  const T* wt = static_cast<const T*>(a.weight);
  float h[CPT][8], w[CPT][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = 8 * (u + i * TPR);
    if (c < a.dim) {
      float r[8] = {};
      load8(x, c, a.dim, h[i]);
      if (res) load8(res, c, a.dim, r);
      if (wt) load8(wt, c, a.dim, w[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[i][e] += r[e];
        ss += h[i][e] * h[i][e];
      }
    }
  }
  if (ro) {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = 8 * (u + i * TPR);
      if (c < a.dim) store8(ro, c, a.dim, h[i]);
    }
  }
  // 1 / sqrt(...) = pre * inv.  From 2^-80 on the squares that 32 bits lose are less than 2^-31 of the sum.
  ss = row_sum<TPR>(ss, s_sum);
  float pre = 1.0f, inv = ss / (float)a.dim + a.eps;
  if (ss >= 0x1p-80f && inv < INFINITY) {
    inv = 1.0f / sqrtf(inv);
  } else {  // the same way for all threads of a row
    double wide = 0.0;
#pragma unroll
    for (int i = 0; i < CPT; ++i)
      if (8 * (u + i * TPR) < a.dim) {
#pragma unroll
        for (int e = 0; e < 8; ++e) wide += (double)h[i][e] * (double)h[i][e];
      }
    wide = row_sum<TPR>(wide, s_wide) / (double)a.dim + (double)a.eps;
    wide = wide == 0.0 ? 0.0 : 1.0 / sqrt(wide);  // a row of zeros without eps gives zeros
    // either factor, and h * pre, stay well inside 32 bits
    pre = wide < 0x1p-64 ? 0x1p-64f : wide > 0x1p64 ? 0x1p64f : 1.0f;
    inv = (float)(wide / (double)pre);
  }
  uint32_t top = 0;  // bits of max|y|: an infinity or a NaN is larger than every number
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = 8 * (u + i * TPR);
    if (c < a.dim) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[i][e] = h[i][e] * pre * inv;
        if (wt) h[i][e] *= w[i][e];
        if (KIND == kNormRow && (c + e < a.dim)) top = max(top, __float_as_uint(h[i][e]) & 0x7fffffffu);
      }
    }
  }
  if constexpr (KIND == kNormSame) {
    T* out = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = 8 * (u + i * TPR);
      if (c < a.dim) store8(out, c, a.dim, h[i]);
    }
  } else {
    uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.out_stride;
    float s = 0.0f, f = 0.0f;
    if (KIND == kNormRow) {
      const float m = __uint_as_float(row_max<TPR>(top, s_max));
      s = m / 448.0f;
      f = 448.0f / m;
      if (u == 0) static_cast<float*>(a.scale)[row] = s;
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = 8 * (u + i * TPR);
      if (KIND == kNormMx) {
        // the four lanes of a block are all inside the row or all behind it: dim is a multiple of 32
        uint32_t m = 0;
        if (c < a.dim) {
#pragma unroll
          for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(h[i][e]) & 0x7fffffffu);
        }
        m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
        // m = 1.f 2^(b - 127) and 448 = 1.75 2^8: s = 2^(b - 135), one more from 1.75 on
        int b = (int)(m >> 23);
        b = b == 255 ? 255 : max(b - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
        if (c < a.dim) {
          if ((u & 3) == 0)
            static_cast<uint8_t*>(a.scale)[row * a.scale_stride + (c >> 5)] = (uint8_t)b;
#pragma unroll
          for (int e = 0; e < 8; ++e) h[i][e] = ldexpf(h[i][e], 127 - b);
        }
      } else if (s > 0x1p-100f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] *= f;
      } else {  // 448 / m may be beyond 32 bits; a row of zeros stays one, NaN stays NaN
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = s == 0.0f ? 0.0f : h[i][e] / s;
      }
      if (c < a.dim) {
        const u32x2 q = pack8_e4m3(h[i]);
        if (c + 8 <= a.dim) {
          *reinterpret_cast<u32x2*>(out + c) = q;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < a.dim) out[c + e] = (uint8_t)(q[e >> 2] >> (8 * (e & 3)));
        }
      }
    }
  }
}

template <typename T, typename R, int KIND>
void launch_kind(const AddNormArgs& a, hipStream_t stream) {
  // a launch takes less than 2^32 threads
  const auto go = [&](auto kernel, int per_block, int threads) {
    constexpr int kSlice = 1 << 21;
    for (int at = 0; at < a.rows; at += kSlice) {
      AddNormArgs s = a;
      const auto on = [&](const void* p, int64_t stride, int es) {
        return p ? (char*)p + (int64_t)at * stride * es : nullptr;
      };
      s.x = on(a.x, a.x_stride, 2);
      s.residual = on(a.residual, a.residual_stride, sizeof(R));
      s.residual_out = on(a.residual_out, a.residual_out_stride, sizeof(R));
      s.out = on(a.out, a.out_stride, KIND == kNormSame ? 2 : 1);
      s.scale = KIND == kNormMx ? on(a.scale, a.scale_stride, 1) : on(a.scale, 1, 4);
      s.rows = a.rows - at < kSlice ? a.rows - at : kSlice;
      PSISPEC_LAUNCH("add_rmsnorm", kernel, dim3((unsigned)((s.rows + per_block - 1) / per_block)), dim3(threads), 0,
                     stream, s);
    }
  };
  // As few threads per row as hold it in 8 or 16 elements each (a wave waits for no other).  In us per launch, BF16
  // with a residual of the same type, three sets of inputs in turn: 8000 x 512 64 threads 9.4, 256 16.5; 8000 x 1024
  // 64 threads 12.5, 256 17.5 (one row 3.5, 3.2); 576 x 4096 256 threads 6.0, 512 6.3 (one row 3.8, 3.4); 576 x 8192
  // 512 threads 10.0, 1024 12.3; 4000 x 16384 1024 threads of 16 elements 99, of up to 32 120.  Where the rows come
  // from memory, not from the cache behind the L2, twice the threads are as fast or faster: 8000 x 4096 256 threads
  // 55.0, 512 51.6 (on one set of 196 MB, which that cache holds, 36.2 and 40.5); 8000 x 8192 512 threads 101, 1024 96
  // (89 and 95).
  if (a.dim <= 512)
    go((k_add_rmsnorm<T, R, KIND, 64, 1>), 4, 256);
  else if (a.dim <= 1024)
    go((k_add_rmsnorm<T, R, KIND, 64, 2>), 4, 256);
  else if (a.dim <= 2048)
    go((k_add_rmsnorm<T, R, KIND, 256, 1>), 1, 256);
  else if (a.dim <= 4096)
    go((k_add_rmsnorm<T, R, KIND, 256, 2>), 1, 256);
  else if (a.dim <= 8192)
    go((k_add_rmsnorm<T, R, KIND, 512, 2>), 1, 512);
  else if (a.dim <= 16384)
    go((k_add_rmsnorm<T, R, KIND, 1024, 2>), 1, 1024);
  else
    go((k_add_rmsnorm<T, R, KIND, 1024, 4>), 1, 1024);
}

template <typename T, typename R>
void launch_types(const AddNormArgs& a, hipStream_t stream) {
  if (a.kind == kNormSame)
    launch_kind<T, R, kNormSame>(a, stream);
  else if (a.kind == kNormRow)
    launch_kind<T, R, kNormRow>(a, stream);
  else
    launch_kind<T, R, kNormMx>(a, stream);
}

}  // namespace

hipError_t launch_add_rmsnorm(const AddNormArgs& a, psispec_dtype dtype, hipStream_t stream) {
  if (dtype == PSISPEC_BF16) {
    if (a.residual_f32)
      launch_types<__bf16, float>(a, stream);
    else
      launch_types<__bf16, __bf16>(a, stream);
  } else {
    if (a.residual_f32)
      launch_types<_Float16, float>(a, stream);
    else
      launch_types<_Float16, _Float16>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace psispec
