// attend.hip -- attention of a block's new tokens over the paged cache.
//
//   out = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale q . k_t) over the positions t that the row sees
#include "paged.h"

namespace psispec {
namespace {

constexpr int kAtThreads = 256;

template <typename T> __device__ inline float cache_f32(const void* p, int64_t i) {
  return (float)static_cast<const T*>(p)[i];
}
struct f8_t {};
template <> __device__ inline float cache_f32<f8_t>(const void* p, int64_t i) {
  return __builtin_amdgcn_cvt_f32_fp8((int)static_cast<const uint8_t*>(p)[i], 0);
}

// One workgroup per (line, block row, query head); each wave takes every fourth position, its lanes
// the dimensions lane, lane + 64, ...
template <typename T, typename C>
__global__ __launch_bounds__(kAtThreads) void k_attend(AttendArgs a) {
  const psispec_paged_cache& c = a.c;
  const int hq = blockIdx.x % a.heads_q;
  const int64_t row = blockIdx.x / a.heads_q;
  const int r = (int)(row / a.blk), i = (int)(row - (int64_t)r * a.blk);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __shared__ uint32_t s_seen[kMaxAttendBlock / 32];
  __shared__ float s_m[4], s_l[4], s_o[4][kMaxHeadDim];
  int L, n;
  const bool ok = line_rows(a.len, a.n_new, r, a.blk, c.slots, c.page_size, &L, &n);
  const int32_t* tab = c.table + (int64_t)r * c.table_stride;
  if (a.status && i == 0 && hq == 0) {
    bool bad = !ok, badp = false;
    if (ok) {
      for (int s = threadIdx.x; (int64_t)s * c.page_size < (int64_t)L + n; s += kAtThreads)
        bad |= (uint32_t)tab[s] >= (uint32_t)c.num_pages;
      if (a.parent)
        for (int j = threadIdx.x; j < n; j += kAtThreads) {
          const int p = a.parent[(int64_t)r * a.blk + j];
          badp |= p < -1 || p >= j;
        }
    }
    const bool b0 = __syncthreads_or(bad), b1 = __syncthreads_or(badp);
    if (threadIdx.x == 0)
      a.status[r] = (b0 ? PSISPEC_ST_BAD_PAGE : 0) | (b1 ? PSISPEC_ST_BAD_PARENT : 0);
  }
  if (!ok || i >= n) return;
  for (int w = threadIdx.x; w < kMaxAttendBlock / 32; w += kAtThreads)
    s_seen[w] = a.parent ? 0u : w < (i >> 5) ? ~0u : w == (i >> 5) ? (2u << (i & 31)) - 1u : 0u;
  __syncthreads();
  if (a.parent && threadIdx.x == 0) {
    int j = i;
    while (j >= 0) {
      s_seen[j >> 5] |= 1u << (j & 31);
      const int p = a.parent[(int64_t)r * a.blk + j];
      j = p < j ? p : -1;
    }
  }
  __syncthreads();
  const int h = hq / (a.heads_q / c.heads);
  const T* q = static_cast<const T*>(a.q) + row * a.q_stride + (int64_t)hq * c.dim;
  float qf[4], o[4] = {};
#pragma unroll
  for (int k = 0; k < 4; ++k) qf[k] = lane + 64 * k < c.dim ? (float)q[lane + 64 * k] : 0.0f;
  const float ks = c.k_scale ? c.k_scale[h] : 1.0f, vs = c.v_scale ? c.v_scale[h] : 1.0f;
  float m = -INFINITY, l = 0.0f;
  for (int t = wave; t < L + i + 1; t += 4) {
    if (t >= L && !((s_seen[(t - L) >> 5] >> ((t - L) & 31)) & 1u)) continue;
    const int slot = t / c.page_size;
    const int page = tab[slot];
    if ((uint32_t)page >= (uint32_t)c.num_pages) continue;
    const int64_t at = (int64_t)page * c.page_stride + (int64_t)(t - slot * c.page_size) * c.row_stride +
                       (int64_t)h * c.head_stride;
    float s = 0.0f, v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool on = lane + 64 * k < c.dim;
      s += on ? qf[k] * cache_f32<C>(c.k, at + lane + 64 * k) : 0.0f;
      v[k] = on ? cache_f32<C>(c.v, at + lane + 64 * k) : 0.0f;
    }
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) s += __shfl_xor(s, x, 64);
    s *= a.scale * ks;
    const float mn = fmaxf(m, s);
    const float f = m == mn ? 1.0f : expf(m - mn), p = expf(s - mn);
    l = l * f + p;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = o[k] * f + p * v[k];
    m = mn;
  }
  if (lane == 0) {
    s_m[wave] = m;
    s_l[wave] = l;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) s_o[wave][lane + 64 * k] = o[k];
  __syncthreads();
  float mx = s_m[0], sum = 0.0f, f[4];
  for (int w = 1; w < 4; ++w) mx = fmaxf(mx, s_m[w]);
  for (int w = 0; w < 4; ++w) {
    f[w] = s_m[w] == -INFINITY ? 0.0f : expf(s_m[w] - mx);
    sum += f[w] * s_l[w];
  }
  T* out = static_cast<T*>(a.out) + row * a.out_stride + (int64_t)hq * c.dim;
  if ((int)threadIdx.x < c.dim) {
    float y = 0.0f;
    for (int w = 0; w < 4; ++w)
      if (s_l[w] != 0.0f) y += f[w] * s_o[w][threadIdx.x];
    out[threadIdx.x] = (T)(y / sum * vs);
  }
}

}  // namespace

size_t attend_workspace_bytes(int, int, int, int, int) { return 256; }

hipError_t launch_attend(const AttendArgs& a, psispec_dtype dtype, void*, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.batch * a.blk * a.heads_q)), block(kAtThreads);
  const bool f8 = a.c.dtype == PSISPEC_F8E4M3;
  if (dtype == PSISPEC_BF16) {
    if (f8)
      PSISPEC_LAUNCH("attend", (k_attend<__bf16, f8_t>), grid, block, 0, stream, a);
    else
      PSISPEC_LAUNCH("attend", (k_attend<__bf16, __bf16>), grid, block, 0, stream, a);
  } else {
    if (f8)
      PSISPEC_LAUNCH("attend", (k_attend<_Float16, f8_t>), grid, block, 0, stream, a);
    else
      PSISPEC_LAUNCH("attend", (k_attend<_Float16, _Float16>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace psispec
