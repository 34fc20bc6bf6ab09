// w4_few.h -- the 4-bit products of few rows, and of more where there are few outputs.
//
// The weights are read once, straight from memory into the registers that feed the matrix cores (the
// packed order makes each load 1 KB in a row).  A workgroup owns NT tiles of 16 outputs; its KW waves take
// the steps of 256 bytes of each row in turn, so that one layer's loads are spread over as many waves as the
// card holds at once, and their sums meet in LDS in the waves' order.  A wave stages the rows of its own
// steps in LDS by loads that write it themselves (whole runs of 256 bytes; straight into the instructions'
// order they would be pieces of 16 bytes), so no wave waits for another before the end.  One step per wave is
// in flight and the waves cover for each other: with two or three the times were the same or worse.
// Bound by the weights' way from memory and, for one layer, by what a launch and its first loads take (4 us).
// In us per launch, in a graph of 42 on three sets of inputs: one row, 6144 x 4096 INT 5.7, 2 x 12288 x 4096 MX gated
// 11 (53 MB, 4.8 TB/s); 9 rows, 4096 x 12288 MX 7.7; 64 rows, 4096 x 4096 INT in F16 8.3 (its waves wait for half of
// their cycles: four steps each, a step's loads waited for before its products), 12288 x 4096 INT 15.3, 2 x 12288 x
// 4096 gated INT 25, MX 21, MX with 8-bit rows 17 (3.2 TB/s: the rows' 98 MB from the L2 beside the weights' 53, and
// one and a half workgroups per CU).  INT tiles of 64 rows need more than the 256 registers that there are: 20 of the
// 24 instantiations keep 2 to 25 values in scratch memory, since the sums of all their tiles live at once.
#pragma once

#include "w4.h"

namespace psispec {
namespace w4 {

// X: __bf16, _Float16 or F8; GPT: INT groups per tile, 0: MX; SF16: INT scales in F16; R4: rows of a workgroup
// over 4
template <typename X, int GPT, bool SF16, int R4, int NT, int MATS, int KW>
__global__ __launch_bounds__(64 * KW, KW < 8 ? 2 : 1) void k_w4_few(W4Args a) {
  constexpr bool kMx = GPT == 0, kF8 = __is_same(X, F8);
  constexpr int MT = R4 < 4 ? 1 : R4 / 4, NB = NT * MATS;
  constexpr int TPS = kF8 ? 2 : 1;                 // tiles of 128 inputs per step
  constexpr int kStage = R4 * 4 * kStageRow;       // bytes of a step's rows
  constexpr int kRead = MT * 16 * kStageRow;       // what the reads of the last stage may reach
  constexpr int kXsAt = KW * kStage + (kRead - kStage);  // 8-bit rows: 512 bytes a wave to turn scales in
  constexpr int kX = kXsAt + (kF8 ? KW * 512 : 0), kAcc = KW * MT * NB * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t s_mem[kX > kAcc ? kX : kAcc];
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int nblocks = (a.ntiles + NT - 1) / NT;
  const int mblock = (int)(blockIdx.x / (unsigned)nblocks);
  const int nt0 = (int)(blockIdx.x - (unsigned)mblock * nblocks) * NT, m0 = mblock * (4 * R4);

  struct Slot {
    u32x4 w[TPS][NB];
    uint32_t e[NB];  // MX: scale byte (8-bit rows: those of both tiles)
    u32x2 s[NB][kMx ? 1 : GPT];
    uint64_t xs;  // 8-bit rows: scales of row `lane`
  };
  Slot q;

  // rows: load i fills rows 4 i .. + 3; slot s of row r holds its 16-byte chunk s ^ (r % 16).  Rows behind the
  // last repeat it and are not stored.
  constexpr int XB = kF8 ? 1 : 2;
  const int rowbytes = a.k * XB, rows = min(4 * R4, a.rows - m0);
  const int stride = (int)a.x_stride * XB;
  const uint8_t* xbase = static_cast<const uint8_t*>(a.x) + (int64_t)m0 * a.x_stride * XB;
  int xoff[R4], chunk[R4];
#pragma unroll
  for (int i = 0; i < R4; ++i) {
    const int r = 4 * i + g;
    chunk[i] = 16 * (c ^ (r & 15));
    xoff[i] = min(r, rows - 1) * stride + chunk[i];
  }
  const uint8_t* xsrow = kF8 ? a.x_scale + (int64_t)(m0 + min(lane, rows - 1)) * a.xs_stride : nullptr;
  const uint8_t *codes[NB], *scales[NB];
  int top[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int nt = min(nt0 + b % NT, a.ntiles - 1);
    codes[b] = a.codes[b / NT] + (int64_t)nt * a.ktiles * 1024;
    scales[b] = static_cast<const uint8_t*>(a.scales[b / NT]) +
                (kMx ? mx_scale_at(nt, 0, a.ktiles) : (int64_t)nt * a.ktiles * (32 * GPT));
    top[b] = 0;
  }
  const uint32_t lane16 = lane * 16;
  uint8_t* const mine = s_mem + wave * kStage;

  const auto load = [&](int st) {
    const int at = st * kStageRow;
    const __amdgpu_buffer_rsrc_t rx =
        __builtin_amdgcn_make_buffer_rsrc((void*)xbase, (short)0, (rows - 1) * stride + rowbytes, kRsrc3);
    if (at + kStageRow <= rowbytes) {
#pragma unroll
      for (int i = 0; i < R4; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(mine + i * 1024), 16, (int)xoff[i], (int)at, 0, 0);
    } else {  // behind the row: zeros
#pragma unroll
      for (int i = 0; i < R4; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(mine + i * 1024), 16,
                                                 (int)(at + chunk[i] < rowbytes ? xoff[i] : 0x7ffffff0),
                                                 min(at, rowbytes), 0, 0);
    }
#pragma unroll
    for (int h = 0; h < TPS; ++h) {
      const int t = min(st * TPS + h, a.ktiles - 1);  // behind the last: any weights will do
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        q.w[h][b] = *reinterpret_cast<const u32x4*>(codes[b] + (int64_t)t * 1024 + lane16);
        if constexpr (kMx) {
          const uint8_t* e = scales[b] + (int64_t)(t / 2) * 128 + (t & 1);
          if (h == 0) q.e[b] = kF8 ? reinterpret_cast<const uint16_t*>(e)[(uint32_t)lane] : e[(uint32_t)(2 * lane)];
        } else {
#pragma unroll
          for (int p = 0; p < GPT; ++p)
            q.s[b][p] = *reinterpret_cast<const u32x2*>(scales[b] + (int64_t)t * (32 * GPT) + 32 * p + (uint32_t)(8 * g));
        }
      }
    }
    if constexpr (kF8) q.xs = row_scales(xsrow, 8 * st, a.k / 32);  // lane = row: a load per row and step
    if (kMx && !kF8 && st == wave) {  // once, behind the first loads (before them: 9 rows, 4096 x 12288 7.7 us instead of 7.4)
#pragma unroll
      for (int b = 0; b < NB; ++b) top[b] = a.top[b / NT][min(nt0 + b % NT, a.ntiles - 1) * 16 + c];
    }
  };

  f32x4 acc[MT][NB];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[m][b] = f32x4{0, 0, 0, 0};

  [[maybe_unused]] const IntBits bits = int_bits<X>();
  const auto read_x = [&](int m, int ch) {
    return lds_read(reinterpret_cast<const u32x4*>(mine + (16 * m + c) * kStageRow + 16 * (ch ^ c)));
  };
  const auto pin = [&] {
#ifdef __HIP_DEVICE_COMPILE__  // the host has no such registers
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int b = 0; b < NB; ++b) asm volatile("" : "+v"(acc[m][b]));
#endif
    __builtin_amdgcn_sched_barrier(0);
  };
  const auto compute = [&] {
    if constexpr (kF8) {
      // lane (row c of a tile, g) takes byte g of either half of the row's scales
      uint64_t* const turn = reinterpret_cast<uint64_t*>(s_mem + kXsAt + wave * 512);
      turn[lane] = q.xs;
      wave_sync();
      uint32_t xs[2][MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const u32x2 v = lds_read(reinterpret_cast<const u32x2*>(turn + 16 * m + c));
        xs[0][m] = v[0] >> (8 * g);
        xs[1][m] = v[1] >> (8 * g);
      }
#pragma unroll
      for (int h = 0; h < TPS; ++h) {
        u32x4 lo[MT], hi[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          lo[m] = read_x(m, 8 * h + g);
          hi[m] = read_x(m, 8 * h + 4 + g);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[m][b] = h == 0 ? mfma_mx<0>(q.w[h][b], (int)q.e[b], lo[m], hi[m], (int)xs[h][m], acc[m][b])
                               : mfma_mx<1>(q.w[h][b], (int)q.e[b], lo[m], hi[m], (int)xs[h][m], acc[m][b]);
      }
    } else if constexpr (kMx) {
      float s[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) s[b] = mx_scale((int)q.e[b], top[b], X());
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 x[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = read_x(m, 4 * g + j);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const u32x4 w = mx_codes(q.w[0][b][j], s[b], X());
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[m][b] = mfma(w, x[m], acc[m][b], X());
        }
      }
    } else {
      constexpr int JG = 4 / GPT;  // instructions per group
#pragma unroll
      for (int p = 0; p < GPT; ++p) {
        f32x4 less[MT], sum[NB][MT];
#pragma unroll
        for (int j = 0; j < JG; ++j) {
          u32x4 x[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            x[m] = read_x(m, 4 * (p * JG + j) + g);
            less[m] = mfma(minus24(X()), x[m], j ? less[m] : f32x4{0, 0, 0, 0}, X());
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const u32x4 w = int_codes(q.w[0][b][p * JG + j], bits, X());
#pragma unroll
            for (int m = 0; m < MT; ++m) sum[b][m] = mfma(w, x[m], j ? sum[b][m] : f32x4{0, 0, 0, 0}, X());
          }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const f32x4 s = scales_of<SF16>(q.s[b][p]);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][b][i] = fmaf(sum[b][m][i] + less[m][i], s[i], acc[m][b][i]);
        }
        pin();  // a group's sums end here: the compiler would start every group's products first
      }
    }
  };

  // A step's place in LDS is loaded again only when its reads are done with (the matrix instructions behind
  // them).
  const int steps = (a.ktiles + TPS - 1) / TPS;
  for (int st = wave; st < steps; st += KW) {
    load(st);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __builtin_amdgcn_sched_barrier(0);
    compute();
    __builtin_amdgcn_sched_barrier(0);
  }

  if constexpr (kMx && __is_same(X, __bf16)) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (__any(top[b] > 252)) {  // the same way for the whole wave
#pragma unroll
        for (int m = 0; m < MT; ++m) mx_back4(acc[m][b], top[b]);
      }
  }
  f32x4(*s_acc)[64] = reinterpret_cast<f32x4(*)[64]>(s_mem);
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int b = 0; b < NB; ++b) s_acc[wave * (MT * NB) + m * NB + b][lane] = acc[m][b];
  __syncthreads();
  for (int o = wave; o < MT * NT; o += KW) {
    const int m = o / NT, b = o - m * NT, n = (nt0 + b) * 16 + 4 * g, row = m0 + 16 * m + c;
    f32x4 y[MATS];
#pragma unroll
    for (int q = 0; q < MATS; ++q) {
      y[q] = s_acc[m * NB + q * NT + b][lane];
#pragma unroll
      for (int w = 1; w < KW; ++w) y[q] += s_acc[w * (MT * NB) + m * NB + q * NT + b][lane];
    }
    if (n >= a.n || row >= a.rows || 16 * m + c >= 4 * R4) continue;
    if constexpr (kMx && __is_same(X, _Float16)) {
#pragma unroll
      for (int q = 0; q < MATS; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[q][i] = mx_back(y[q][i], a.top[q][n + i], X());
    }
    store4<MATS>(a, row, n, y[0], y[MATS - 1]);
  }
}

template <typename X, int GPT, bool SF16, int MATS>
hipError_t launch_few_scales(const W4Args& a, hipStream_t stream) {
  constexpr int kWide = MATS == 2 ? 2 : 4;
  const FewPlan p = few_plan(a.rows, a.ntiles, a.ktiles, MATS);
  const auto go = [&](auto kernel) {
    PSISPEC_LAUNCH(MATS == 2 ? "w4_gated" : "w4_linear", kernel, dim3((unsigned)p.blocks), dim3(64 * p.kw), 0, stream,
                   a);
  };
  if (p.r4 == 16 && p.kw == 4) {
    go((k_w4_few<X, GPT, SF16, 16, kWide, MATS, 4>));
  } else if (p.r4 == 16) {
    go((k_w4_few<X, GPT, SF16, 16, kWide, MATS, 8>));
  } else if (p.r4 == 8 && p.nt == 4) {
    if constexpr (MATS == 1) {
      if (p.kw == 4)
        go((k_w4_few<X, GPT, SF16, 8, 4, MATS, 4>));
      else
        go((k_w4_few<X, GPT, SF16, 8, 4, MATS, 8>));
    }
  } else if (p.r4 == 8 && p.kw == 4) {
    go((k_w4_few<X, GPT, SF16, 8, 2, MATS, 4>));
  } else if (p.r4 == 8) {
    go((k_w4_few<X, GPT, SF16, 8, 2, MATS, 8>));
  } else if (p.r4 == 4 && p.nt == 2) {
    go((k_w4_few<X, GPT, SF16, 4, 2, MATS, 8>));
  } else if (p.r4 == 4 && p.kw == 16) {
    go((k_w4_few<X, GPT, SF16, 4, 1, MATS, 16>));
  } else if (p.r4 == 4) {
    go((k_w4_few<X, GPT, SF16, 4, 1, MATS, 8>));
  } else if (p.kw == 16) {
    go((k_w4_few<X, GPT, SF16, 1, 1, MATS, 16>));
  } else {
    go((k_w4_few<X, GPT, SF16, 1, 1, MATS, 8>));
  }
  return hipGetLastError();
}

template <typename X, int GPT, int MATS>
hipError_t launch_few(const W4Args& a, hipStream_t stream) {
  if constexpr (GPT > 0)
    if (a.scale_f16) return launch_few_scales<X, GPT, true, MATS>(a, stream);
  return launch_few_scales<X, GPT, false, MATS>(a, stream);
}

}  // namespace w4
}  // namespace psispec
