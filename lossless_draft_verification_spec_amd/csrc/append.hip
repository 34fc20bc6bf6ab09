// append.hip -- the block's queries, keys and values: norm, position rotation, and K and V into pages.
//
//   x = x / sqrt(mean(x^2) + eps) * w           per query / key head, when it has a weight
//   (a, b) = s (a cos t - b sin t, b cos t + a sin t), t = position * f_j, pairs j of the first rot
//   dimensions: (j, j + rot/2) or (2j, 2j + 1)
//
// One workgroup per token row.  The cosines and sines are the same for all heads of a row, so they
// are formed once, in LDS: t in fp64 (a position of 10^6 times a frequency of 1 would be off by 0.06
// in fp32), reduced to a turn in fp64, sin and cos of the turn in fp32 (absolute error 2e-7, far
// below the 16-bit output's rounding).  A head of D dimensions belongs to D/16 lanes; a lane holds
// two 8-element chunks, those of one run of pairs (c, c + rot/16) in the half layout, so a rotation
// needs no exchange between lanes and q may be rotated in place.  Bound by HBM for many rows (every
// input element read once, every output written once), by the chain len -> table -> store for few.
// 32 query and 8 key/value heads of 128: 8000 rows 40 us (4.9 TB/s, a large copy reaches 4.75), 2304 rows
// of which 1920 live into an 8-bit cache 15 us (3.1 TB/s), 9 rows 5.2 us.
#include "paged.h"

namespace psispec {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

template <typename T> struct Vec8;
template <> struct Vec8<__bf16> { typedef bf16x8 type; };
template <> struct Vec8<_Float16> { typedef f16x8 type; };

constexpr int kAppendThreads = 256;  // 512, one pass over 48 heads: 8000 rows 45 us instead of 40

__device__ inline float clamp_e4m3(float x) {
  const float y = fminf(fmaxf(x, -448.0f), 448.0f);
  return x == x ? y : x;  // NaN stays
}

// 8 values, rounded to nearest, to 8 bytes
__device__ inline u32x2 pack_e4m3(const float* x) {
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int u = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
    u = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], u, true);
    w[i] = (uint32_t)u;
  }
  return w;
}

// T: element type of the inputs; F8: the cache holds 8-bit numbers, else T.  log_group: lanes of a head,
// D/16 rounded up to a power of two.
template <typename T, bool F8>
__global__ __launch_bounds__(kAppendThreads) void k_qkv_append(AppendArgs a, int log_group) {
  typedef typename Vec8<T>::type V8;
  __shared__ float s_cos[kMaxHeadDim / 2], s_sin[kMaxHeadDim / 2];
  const psispec_paged_cache& c = a.c;
  const int64_t row = blockIdx.x;
  const int r = (int)(row / a.blk), i = (int)(row - (int64_t)r * a.blk);
  const int rot = a.p.rot, half = rot >> 1;
  const int group = 1 << log_group;
  const int u = threadIdx.x & (group - 1);
  const bool lane_on = u < (c.dim >> 4);
  // the lane's two chunks of 8 dimensions
  const int rp = rot >> 4;               // lanes that hold rotated pairs
  const bool rotated = u < rp;
  const bool inter = (a.p.flags & PSISPEC_ROPE_INTERLEAVED) != 0;
  int c0 = 2 * u, c1 = 2 * u + 1;
  if (rotated && !inter) {
    c0 = u;
    c1 = u + rp;
  }
  const int heads = a.heads_q + 2 * c.heads, per_pass = kAppendThreads >> log_group;
  const int hd0 = threadIdx.x >> log_group;

  // The first heads and the frequency do not hang on the line's length: they are on their way during
  // the chain length -> page -> place.
  auto load = [&](int hd, V8& raw0, V8& raw1) {
    const int kind = hd < a.heads_q ? 0 : hd < a.heads_q + c.heads ? 1 : 2;  // q, k, v
    const int h = kind == 0 ? hd : kind == 1 ? hd - a.heads_q : hd - a.heads_q - c.heads;
    const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                   row * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) +
                   (int64_t)h * c.dim;
    raw0 = *reinterpret_cast<const V8*>(src + 8 * c0);
    raw1 = *reinterpret_cast<const V8*>(src + 8 * c1);
  };
  V8 raw0 = {}, raw1 = {};
  if (lane_on && hd0 < heads) load(hd0, raw0, raw1);
  const double freq = (int)threadIdx.x < half ? a.p.inv_freq[threadIdx.x] : 0.0;

  int L, n;
  const bool ok = line_rows(a.len, a.n_new, r, a.blk, c.slots, c.page_size, &L, &n);
  const int32_t* tab = c.table + (int64_t)r * c.table_stride;
  if (i == 0 && a.status) {  // row 0's workgroup reports for its line
    bool bad = !ok;
    if (ok && n > 0) {
      const int s0 = L / c.page_size, s1 = (L + n - 1) / c.page_size;
      for (int s = s0 + (int)threadIdx.x; s <= s1; s += kAppendThreads)
        bad |= (uint32_t)tab[s] >= (uint32_t)c.num_pages;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) a.status[r] = bad ? PSISPEC_ST_BAD_PAGE : 0;
  }
  if (!ok || i >= n) return;
  const int slot = (L + i) / c.page_size, off = (L + i) - slot * c.page_size;
  const int page = tab[slot];
  if ((uint32_t)page >= (uint32_t)c.num_pages) return;
  const int pos = a.positions ? a.positions[row] : L + i;
  if ((int)threadIdx.x < half) {  // half <= 128
    const double t = (double)pos * freq * 0.15915494309189533577;  // turns
    float sn, cs;
    sincospif(2.0f * (float)(t - rint(t)), &sn, &cs);
    s_cos[threadIdx.x] = cs * (float)a.p.rope_scale;
    s_sin[threadIdx.x] = sn * (float)a.p.rope_scale;
  }
  __syncthreads();

  const int64_t at = (int64_t)page * c.page_stride + (int64_t)off * c.row_stride;
  const float eps = (float)a.p.eps, inv_d = 1.0f / (float)c.dim;
  for (int hd = hd0; hd < heads; hd += per_pass) {
    if (hd != hd0 && lane_on) load(hd, raw0, raw1);
    const int kind = hd < a.heads_q ? 0 : hd < a.heads_q + c.heads ? 1 : 2;
    const int h = kind == 0 ? hd : kind == 1 ? hd - a.heads_q : hd - a.heads_q - c.heads;
    float x[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[0][e] = (float)raw0[e];
      x[1][e] = (float)raw1[e];
    }
    if (kind < 2) {
      const T* w = static_cast<const T*>(kind == 0 ? a.p.q_weight : a.p.k_weight);
      if (w) {
        V8 w0 = {}, w1 = {};
        if (lane_on) {
          w0 = *reinterpret_cast<const V8*>(w + 8 * c0);
          w1 = *reinterpret_cast<const V8*>(w + 8 * c1);
        }
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += x[0][e] * x[0][e] + x[1][e] * x[1][e];
        for (int o = 1; o < group; o <<= 1) ss += __shfl_xor(ss, o, 64);
        const float inv = 1.0f / sqrtf(ss * inv_d + eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[0][e] *= inv * (float)w0[e];
          x[1][e] *= inv * (float)w1[e];
        }
      }
      if (rotated) {
        if (!inter) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float cs = s_cos[8 * u + e], sn = s_sin[8 * u + e];
            const float p = x[0][e], z = x[1][e];
            x[0][e] = p * cs - z * sn;
            x[1][e] = z * cs + p * sn;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {  // pairs 8u + e of the lane's 16 dimensions
            const float cs = s_cos[8 * u + e], sn = s_sin[8 * u + e];
            const float p = x[e >> 2][(2 * e) & 7], z = x[e >> 2][(2 * e + 1) & 7];
            x[e >> 2][(2 * e) & 7] = p * cs - z * sn;
            x[e >> 2][(2 * e + 1) & 7] = z * cs + p * sn;
          }
        }
      }
    }
    if (!lane_on) continue;
    if (kind > 0 && F8) {
      const float* sc = kind == 1 ? c.k_scale : c.v_scale;
      const float s = sc ? sc[h] : 1.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[0][e] = clamp_e4m3(x[0][e] / s);
        x[1][e] = clamp_e4m3(x[1][e] / s);
      }
      uint8_t* dst = static_cast<uint8_t*>(kind == 1 ? c.k : c.v) + at + (int64_t)h * c.head_stride;
      if (c1 == c0 + 1) {
        const u32x2 lo = pack_e4m3(x[0]), hi = pack_e4m3(x[1]);
        *reinterpret_cast<u32x4*>(dst + 8 * c0) = u32x4{lo[0], lo[1], hi[0], hi[1]};
      } else {
        *reinterpret_cast<u32x2*>(dst + 8 * c0) = pack_e4m3(x[0]);
        *reinterpret_cast<u32x2*>(dst + 8 * c1) = pack_e4m3(x[1]);
      }
      continue;
    }
    T* dst = kind == 0 ? static_cast<T*>(a.q_out) + row * a.q_out_stride + (int64_t)h * c.dim
                       : static_cast<T*>(kind == 1 ? c.k : c.v) + at + (int64_t)h * c.head_stride;
    if (kind < 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        raw0[e] = (T)x[0][e];
        raw1[e] = (T)x[1][e];
      }
    }
    *reinterpret_cast<V8*>(dst + 8 * c0) = raw0;
    *reinterpret_cast<V8*>(dst + 8 * c1) = raw1;
  }
}

}  // namespace

hipError_t launch_qkv_append(const AppendArgs& a, psispec_dtype dtype, hipStream_t stream) {
  int lg = 0;
  while ((1 << lg) < a.c.dim / 16) ++lg;
  const dim3 grid((unsigned)((int64_t)a.batch * a.blk));
  const bool f8 = a.c.dtype == PSISPEC_F8E4M3;
  if (dtype == PSISPEC_BF16) {
    if (f8)
      PSISPEC_LAUNCH("qkv_append", (k_qkv_append<__bf16, true>), grid, dim3(kAppendThreads), 0,
                     stream, a, lg);
    else
      PSISPEC_LAUNCH("qkv_append", (k_qkv_append<__bf16, false>), grid, dim3(kAppendThreads), 0,
                     stream, a, lg);
  } else {
    if (f8)
      PSISPEC_LAUNCH("qkv_append", (k_qkv_append<_Float16, true>), grid, dim3(kAppendThreads), 0,
                     stream, a, lg);
    else
      PSISPEC_LAUNCH("qkv_append", (k_qkv_append<_Float16, false>), grid, dim3(kAppendThreads), 0,
                     stream, a, lg);
  }
  return hipGetLastError();
}

}  // namespace psispec
