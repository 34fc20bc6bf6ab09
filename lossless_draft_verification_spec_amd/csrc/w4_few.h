// w4_few.h -- the 4-bit products of few rows.
//
// The weights are read once, straight from memory into the registers that feed the matrix cores (the
// packed order makes each load 1 KB in a row); the rows' operands come from the L2.  A workgroup owns
// NT tiles of 16 outputs and MT of 16 rows; its KW waves take the tiles of 128 inputs in turn, so that
// one layer's worth of loads is spread over as many waves as the card holds at once, and their sums meet
// in LDS in the waves' order.  Each wave keeps the loads of D tiles in flight.
#pragma once

#include "w4.h"

namespace psispec {
namespace w4 {

// X: __bf16, _Float16 or F8; GPT: INT groups per tile, 0: MX
template <typename X, int GPT, int MT, int NT, int MATS, int KW, int D>
__global__ __launch_bounds__(64 * KW) void k_w4_few(W4Args a) {
  constexpr bool kMx = GPT == 0, kF8 = __is_same(X, F8);
  constexpr int NB = NT * MATS, XL = kF8 ? 2 : 4;
  __shared__ f32x4 s_acc[KW][MT * NB][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int nblocks = (a.ntiles + NT - 1) / NT;
  const int mblock = (int)(blockIdx.x / (unsigned)nblocks);
  const int nt0 = (int)(blockIdx.x - (unsigned)mblock * nblocks) * NT, m0 = mblock * (16 * MT);

  struct Slot {
    u32x4 w[NB];
    u32x4 x[MT][XL];
    uint32_t e[NB];  // MX: scale byte
    u32x2 s[NB][kMx ? 1 : GPT];
    uint32_t xs[MT];
  };
  Slot slot[D];

  const uint8_t* xrow[MT];
  const uint8_t* xsrow[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = min(m0 + 16 * m + c, a.rows - 1);  // rows behind the last repeat it and are not stored
    xrow[m] = static_cast<const uint8_t*>(a.x) + (int64_t)row * a.x_stride * (kF8 ? 1 : 2);
    xsrow[m] = kF8 ? a.x_scale + (int64_t)row * a.xs_stride : nullptr;
  }
  int top[NB];
  if constexpr (kMx && !kF8) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
      top[b] = __is_same(X, _Float16) ? a.top[b / NT][min(nt0 + b % NT, a.ntiles - 1) * 16 + c] : 0;
  }

  const auto load = [&](Slot& q, int t) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int64_t tile = (int64_t)min(nt0 + b % NT, a.ntiles - 1) * a.ktiles + t;
      q.w[b] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4*>(a.codes[b / NT] + tile * 1024 + lane * 16));
      if constexpr (kMx)
        q.e[b] = static_cast<const uint8_t*>(a.scales[b / NT])[tile * 64 + lane];
#pragma unroll
      for (int p = 0; p < GPT; ++p)
        q.s[b][p] = static_cast<const u32x2*>(a.scales[b / NT])[(tile * GPT + p) * 4 + g];
    }
    const bool whole = (t + 1) * 128 <= a.k;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if constexpr (kF8) {
        const int blk = 4 * t + g;
        q.xs[m] = whole || blk * 32 < a.k ? xsrow[m][blk] : 127;
      }
#pragma unroll
      for (int j = 0; j < XL; ++j) {
        const int k = t * 128 + (kF8 ? 32 * g + 16 * j : kMx ? 32 * g + 8 * j : 32 * j + 8 * g);
        q.x[m][j] = whole || k < a.k ? *reinterpret_cast<const u32x4*>(xrow[m] + k * (kF8 ? 1 : 2))
                                     : u32x4{0, 0, 0, 0};
      }
    }
  };

  f32x4 acc[MT][NB];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[m][b] = f32x4{0, 0, 0, 0};

  [[maybe_unused]] const IntBits bits = int_bits<X>();
  const auto compute = [&](const Slot& q) {
    if constexpr (kF8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 x[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
          x[m] = f8_rows(q.x[m][j >> 1][2 * (j & 1)], q.x[m][j >> 1][2 * (j & 1) + 1],
                         __uint_as_float(q.xs[m] << 23));
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const u32x4 w = mx_codes(q.w[b][j], __uint_as_float(q.e[b] << 23), __bf16());
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[m][b] = mfma(w, x[m], acc[m][b], __bf16());
        }
      }
    } else if constexpr (kMx) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float s = mx_scale((int)q.e[b], top[b], X());
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 w = mx_codes(q.w[b][j], s, X());
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[m][b] = mfma(w, q.x[m][j], acc[m][b], X());
        }
      }
    } else {
      constexpr int JG = 4 / GPT;  // instructions per group
#pragma unroll
      for (int p = 0; p < GPT; ++p) {
        f32x4 first[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          first[m] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < JG; ++j) first[m] = mfma(minus24(X()), q.x[m][p * JG + j], first[m], X());
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const f32x4 s = a.scale_f16 ? scales_of<true>(q.s[b][p]) : scales_of<false>(q.s[b][p]);
          f32x4 part[MT];
#pragma unroll
          for (int j = 0; j < JG; ++j) {
            const u32x4 w = int_codes(q.w[b][p * JG + j], bits, X());
#pragma unroll
            for (int m = 0; m < MT; ++m) part[m] = mfma(w, q.x[m][p * JG + j], j ? part[m] : first[m], X());
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][b][i] = fmaf(part[m][i], s[i], acc[m][b][i]);
        }
      }
    }
  };

#pragma unroll
  for (int d = 0; d < D; ++d)
    if (wave + d * KW < a.ktiles) load(slot[d], wave + d * KW);
  for (int t = wave; t < a.ktiles; t += KW * D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (t + d * KW < a.ktiles) compute(slot[d]);
      if (t + (d + D) * KW < a.ktiles) load(slot[d], t + (d + D) * KW);
    }
  }

#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int b = 0; b < NB; ++b) s_acc[wave][m * NB + b][lane] = acc[m][b];
  __syncthreads();
  for (int o = wave; o < MT * NT; o += KW) {
    const int m = o / NT, b = o - m * NT, n = (nt0 + b) * 16 + 4 * g, row = m0 + 16 * m + c;
    f32x4 y[MATS];
#pragma unroll
    for (int q = 0; q < MATS; ++q) {
      y[q] = s_acc[0][m * NB + q * NT + b][lane];
      for (int w = 1; w < KW; ++w) y[q] += s_acc[w][m * NB + q * NT + b][lane];
    }
    if (n >= a.n || row >= a.rows) continue;
    if constexpr (kMx && __is_same(X, _Float16)) {
#pragma unroll
      for (int q = 0; q < MATS; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[q][i] = mx_back(y[q][i], a.top[q][n + i], X());
    }
    store4<MATS>(a, row, n, y[0], y[MATS - 1]);
  }
}

template <typename X, int GPT, int MATS>
hipError_t launch_few(const W4Args& a, hipStream_t stream) {
  const auto go = [&](auto kernel, int mt, int nt, int kw) {
    const dim3 grid((unsigned)((a.ntiles + nt - 1) / nt) * (unsigned)((a.rows + 16 * mt - 1) / (16 * mt)));
    PSISPEC_LAUNCH(MATS == 2 ? "w4_gated" : "w4_linear", kernel, grid, dim3(64 * kw), 0, stream, a);
  };
  if (a.rows <= 16)
    go((k_w4_few<X, GPT, 1, 1, MATS, 8, 4>), 1, 1, 8);
  else if (a.rows <= 32)
    go((k_w4_few<X, GPT, 2, 1, MATS, 8, 2>), 2, 1, 8);
  else
    go((k_w4_few<X, GPT, 4, 2, MATS, 4, 1>), 4, 2, 4);
  return hipGetLastError();
}

}  // namespace w4
}  // namespace psispec
