// w4_many.h -- the 4-bit products of many rows.
//
// A workgroup of four waves owns 64 rows x 64 NB outputs of all matrices, a wave 64 rows x 16 NB outputs.  The
// rows go through LDS, 256 bytes of each per step, by loads that write LDS themselves; slot s of row r holds the
// row's 16-byte chunk s ^ (r % 16), so that the reads of 16 rows at one chunk fall on all banks.  The weights come
// straight from memory in the order of the matrix instructions and are decoded once per 64 rows.  What INT
// products start from, -24 sum(x) per row and group, is formed by one pass over the rows before (k_w4_sums) and
// travels with them: formed by the matrix cores here it would be a fifth of their work.  Loads run one step
// ahead (two steps, 576 rows, 12288 x 4096: 8-bit rows 37 us instead of 35, MX 59 and 59; 128 rows per workgroup
// were no faster either).  Few tiles: the inputs are cut into parts whose sums are joined in their order by k_w4_join.
// In us per launch, in a graph of 42 on three sets of inputs: 576 rows, 12288 x 4096: INT 64 (0.90 PFLOP/s), MX 53
// (1.1), MX with 8-bit rows 33 (1.8); two such INT layers gated 123; 2048 rows, 4096 x 12288: 187 (1.10), 157 (1.31),
// 86 (2.4); a library product of 16-bit numbers takes 184 for the last.  INT scales per 64 and per 32 inputs: 211 and
// 254 instead of 187 (two and four times the scales' products).  INT is bound by the vector units beside the matrix
// cores (decoding, scales: four instructions of theirs per matrix instruction, which keeps them as long as it takes
// itself; their order within a tile made no difference).  With 8-bit rows and 432 workgroups (576 rows, 6144 x 4096)
// it is the wait for each step's loads: the waves wait for 0.36 of their cycles, the matrix units are busy for 0.35
// and LDS for 0.23 of them, and 80 CUs hold one workgroup instead of two.
#pragma once

#include "w4.h"

namespace psispec {
namespace w4 {

constexpr int kBM = 64;  // rows of a workgroup

struct ManyArgs {
  W4Args a;
  float* sums;  // INT: [tile of inputs][group][rows up to a multiple of 64]
  float* part;  // cut inputs: [part][matrix][row][output, up to a multiple of 16]
  int mpad, npad, mblocks, nblocks, parts, steps;  // steps of a part
  int band;                                        // row blocks of a band
};

// -24 sum(x) over each group of each row: 16 lanes per row and run of kSumTiles tiles of 128 inputs, 8 inputs of
// each, all read before the first is summed.  Bound by the rows' bytes: 2048 rows of 12288 10.6 us (one tile at a time
// 12.5), 8000 rows 43 (53).
constexpr int kSumTiles = 4;
template <typename X>
__global__ __launch_bounds__(256) void k_w4_sums(ManyArgs m) {
  const W4Args& a = m.a;
  const int c = threadIdx.x & 15, per = 16 / a.gpt;  // lanes of a group
  const int64_t all = (int64_t)m.mpad * ((a.ktiles + kSumTiles - 1) / kSumTiles);
  for (int64_t item = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); item < all; item += (int64_t)gridDim.x * 16) {
    const int t0 = (int)(item / m.mpad) * kSumTiles, row = (int)(item % m.mpad), k = t0 * 128 + 8 * c;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + (int64_t)row * a.x_stride + k;
    u32x4 v[kSumTiles];
#pragma unroll
    for (int i = 0; i < kSumTiles; ++i)  // what is not there: the first row's start, without a branch
      v[i] = *reinterpret_cast<const u32x4*>(row < a.rows && k + 128 * i < a.k ? (const void*)(x + 128 * i) : a.x);
#pragma unroll
    for (int i = 0; i < kSumTiles; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s += scale16(v[i][j] & 0xffffu, __is_same(X, _Float16)) + scale16(v[i][j] >> 16, __is_same(X, _Float16));
      s = row < a.rows && k + 128 * i < a.k ? s : 0.0f;
      for (int o = 1; o < per; o <<= 1) s += __shfl_xor(s, o, 64);  // mpad is a multiple of 64: whole waves
      if (c % per == 0 && t0 + i < a.ktiles) m.sums[((int64_t)(t0 + i) * a.gpt + c / per) * m.mpad + row] = -24.0f * s;
    }
  }
}

// The parts' sums in their order, then what a product ends with; a thread per four outputs.
template <int MATS>
__global__ __launch_bounds__(256) void k_w4_join(ManyArgs m) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, plane = (int64_t)m.a.rows * m.npad;
  if (4 * i >= plane) return;
  const int64_t row = 4 * i / m.npad;
  const int n = (int)(4 * i - row * m.npad);
  if (n >= m.a.n) return;
  f32x4 y[MATS];
#pragma unroll
  for (int q = 0; q < MATS; ++q) {
    y[q] = *reinterpret_cast<const f32x4*>(m.part + q * plane + 4 * i);
    for (int p = 1; p < m.parts; ++p)
      y[q] += *reinterpret_cast<const f32x4*>(m.part + ((int64_t)p * MATS + q) * plane + 4 * i);
  }
  store4<MATS>(m.a, row, n, y[0], y[MATS - 1]);
}

// X: __bf16, _Float16 or F8; GPT: INT groups per tile, 0: MX; SF16: scales in F16
// NB: tiles of 16 outputs of a wave, of all matrices
template <typename X, int GPT, int MATS, bool SF16, int NB>
__global__ __launch_bounds__(256, 2) void k_w4_many(ManyArgs m) {
  constexpr bool kMx = GPT == 0, kF8 = __is_same(X, F8);
  constexpr int MT = kBM / 16, NT = NB / MATS, kLoads = kBM / 16;
  constexpr int TPS = kF8 ? 2 : 1;  // tiles of 128 inputs per step
  // One array: rows, then (INT) -24 sum(x) [group][row], then the scales of each wave's tiles [tile][group][16
  // outputs].  With several arrays the compiler gives each an alias scope and waits for their loads again.
  constexpr int kSumAt = kBM * kStageRow, kScAt = kSumAt + (kF8 ? 4 * 512 : kMx ? 0 : GPT * kBM * 4);
  constexpr int kScLoads = (NB * 8 * GPT + 63) / 64;  // words of a wave's scales over 64
  constexpr int kScWave = kMx ? 0 : kScLoads * 256, kStage = kScAt + 4 * kScWave;
  __shared__ __attribute__((aligned(1024))) uint8_t s_x[2][kStage];
  const W4Args& a = m.a;
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));

  // Neighbouring workgroups go to the eight XCDs in turn: each XCD gets a run of tiles in bands of about eight
  // row blocks, within a band column by column.  The 64 tiles that an XCD holds at once are then about eight row
  // blocks x eight columns, which share rows and weights in its L2 (without bands 8000 rows, 4096 x 12288: INT
  // 733 us instead of 695; 2048 rows, 12288 x 4096 gated: 387 instead of 368; 4096 x 12288 MX 177 instead of 168).
  const unsigned total = (unsigned)m.mblocks * m.nblocks * m.parts, per = total / 8, rest = total % 8;
  const unsigned xcd = blockIdx.x & 7, in = blockIdx.x >> 3;
  const unsigned id = xcd * per + (xcd < rest ? xcd : rest) + in;
  const unsigned plane = (unsigned)m.mblocks * m.nblocks, in_plane = id % plane, band = (unsigned)m.band * m.nblocks;
  const int part = (int)(id / plane), first = (int)(in_plane / band) * m.band, high = min(m.band, m.mblocks - first);
  const int mb = first + (int)(in_plane % band % high), nb = (int)(in_plane % band / high);
  const int m0 = mb * kBM;
  const int nt0 = (nb * 4 + wave) * NT;
  const int step0 = part * m.steps, step1 = min(step0 + m.steps, (a.ktiles + TPS - 1) / TPS);

  // rows into LDS: load i of a wave fills four rows from 4 (kLoads wave + i) on
  const int rowbytes = a.k * (kF8 ? 1 : 2);
  const int rows = min(kBM, a.rows - m0);
  const int64_t stride = a.x_stride * (kF8 ? 1 : 2);
  const uint8_t* xbase = static_cast<const uint8_t*>(a.x) + (int64_t)m0 * stride;
  const int extent = (int)((rows - 1) * stride) + rowbytes;
  int off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = 4 * (kLoads * wave + i) + (lane >> 4);
    off[i] = (int)(min(r, rows - 1) * stride) + 16 * ((lane & 15) ^ (r & 15));
  }
  // word `lane` of load i of a tile's scales: pairs of outputs, 8 GPT words a tile (lanes behind the
  // last repeat the first)
  const uint32_t* sc_at[kMx ? 1 : kScLoads];
  if constexpr (!kMx) {
#pragma unroll
    for (int i = 0; i < kScLoads; ++i) {
      const int word = (64 * i + lane) % (NB * 8 * GPT), b = word / (8 * GPT);
      const int64_t tile = (int64_t)min(nt0 + b % NT, a.ntiles - 1) * a.ktiles;
      sc_at[i] = static_cast<const uint32_t*>(b / NT ? a.scales[1] : a.scales[0]) + tile * (8 * GPT) + word % (8 * GPT);
    }
  }
  const auto load_x = [&](int st, int buf) {
    const int at = st * kStageRow;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)(xbase + at), (short)0, extent - at, kRsrc3);
    const bool whole = at + kStageRow <= rowbytes;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int rr = 4 * (kLoads * wave + i) + (lane >> 4);
      const int o = whole || at + 16 * ((lane & 15) ^ (rr & 15)) < rowbytes ? off[i] : 0x7ffffff0;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(s_x[buf] + 4 * (kLoads * wave + i) * kStageRow), 16, (int)o, 0, 0,
                                               0);
    }
    if constexpr (!kMx) {
      // its 64 rows of a group each wave (with fewer groups than waves some load the same)
      const int grp = wave % GPT;
      __builtin_amdgcn_global_load_lds(
          (const global_u32*)(m.sums + ((int64_t)st * GPT + grp) * m.mpad + m0 + lane),
          (lds_void*)(s_x[buf] + kSumAt + 4 * kBM * grp), 4, 0, 0);
#pragma unroll
      for (int i = 0; i < kScLoads; ++i)
        __builtin_amdgcn_global_load_lds((const global_u32*)(sc_at[i] + (int64_t)st * (8 * GPT)),
                                         (lds_void*)(s_x[buf] + kScAt + wave * kScWave + 256 * i), 4, 0, 0);
    }
  };

  struct Codes {
    uint64_t xs;  // 8-bit rows: scales of row `lane`
    u32x4 w[TPS][NB];
    uint32_t e[NB];  // MX: scale byte (8-bit rows: those of both tiles)
  };
  const uint8_t* xsrow = kF8 ? a.x_scale + (int64_t)min(m0 + lane, a.rows - 1) * a.xs_stride : nullptr;
  int top[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
    top[b] = kMx && !kF8 ? a.top[b / NT][min(nt0 + b % NT, a.ntiles - 1) * 16 + c] : 0;
  const auto load_w = [&](Codes& q, int st) {
#pragma unroll
    for (int h = 0; h < TPS; ++h) {
      const int t = min(st * TPS + h, a.ktiles - 1);  // behind the last: rows of zeros, any weights will do
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int nt = min(nt0 + b % NT, a.ntiles - 1);
        const int64_t tile = (int64_t)nt * a.ktiles + t;
        q.w[h][b] = *reinterpret_cast<const u32x4*>(a.codes[b / NT] + tile * 1024 + lane * 16);
        if (kMx && h == 0) {
          const uint8_t* e = static_cast<const uint8_t*>(a.scales[b / NT]) + mx_scale_at(nt, t, a.ktiles);
          q.e[b] = kF8 ? reinterpret_cast<const uint16_t*>(e)[lane] : e[2 * lane];
        }
      }
    }
    if constexpr (kF8) {
      q.xs = row_scales(xsrow, 8 * st, a.k / 32);  // lane = row: a load per row and step, not per operand
    }
  };

  f32x4 acc[MT][NB];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[i][b] = f32x4{0, 0, 0, 0};

  // the wave's row 16 i + c at chunk `ch`
  const auto read_x = [&](int buf, int i, int ch) {
    return lds_read(reinterpret_cast<const u32x4*>(s_x[buf] + (16 * i + c) * kStageRow + 16 * (ch ^ c)));
  };
  [[maybe_unused]] const IntBits bits = int_bits<X>();
  const auto compute = [&](const Codes& q, int buf) {
    if constexpr (kF8) {
      // each wave turns the rows' scales for itself: lane (row c of a tile, g) takes byte g of either half
      uint64_t* const mine = reinterpret_cast<uint64_t*>(s_x[buf] + kSumAt + wave * 512);
      mine[lane] = q.xs;
      wave_sync();
      uint32_t xs[2][MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const u32x2 v = lds_read(reinterpret_cast<const u32x2*>(mine + 16 * i + c));
        xs[0][i] = v[0] >> (8 * g);
        xs[1][i] = v[1] >> (8 * g);
      }
#pragma unroll
      for (int h = 0; h < TPS; ++h) {
        u32x4 lo[MT], hi[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          lo[i] = read_x(buf, i, 8 * h + g);
          hi[i] = read_x(buf, i, 8 * h + 4 + g);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < MT; ++i)
            acc[i][b] = h == 0 ? mfma_mx<0>(q.w[h][b], (int)q.e[b], lo[i], hi[i], (int)xs[h][i], acc[i][b])
                               : mfma_mx<1>(q.w[h][b], (int)q.e[b], lo[i], hi[i], (int)xs[h][i], acc[i][b]);
      }
    } else if constexpr (kMx) {
      float s[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#ifdef __HIP_DEVICE_COMPILE__
        asm volatile("" : "+v"(top[b]));  // looked at here: before the loop it would be waited for
#endif
        s[b] = mx_scale((int)q.e[b], top[b], X());
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 x[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) x[i] = read_x(buf, i, 4 * g + j);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const u32x4 w = mx_codes(q.w[0][b][j], s[b], X());
#pragma unroll
          for (int i = 0; i < MT; ++i) acc[i][b] = mfma(w, x[i], acc[i][b], X());
        }
      }
    } else {
      // A group's products with one tile of outputs, then, under the next ones, its sums times the scales: the
      // barriers keep the compiler from starting every group's products first (it would spill 200 registers).
      constexpr int JG = 4 / GPT;
      f32x4 sum[2][MT], s[2];
      const auto scale_in = [&](int at, int b) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][b][e] = fmaf(sum[at][i][e], s[at][e], acc[i][b][e]);
      };
#pragma unroll
      for (int p = 0; p < GPT; ++p) {
        u32x4 x[JG][MT];
        f32x4 first[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const float f = lds_read(reinterpret_cast<const float*>(s_x[buf] + kSumAt) + p * kBM + 16 * i + c);
          first[i] = f32x4{f, f, f, f};
#pragma unroll
          for (int j = 0; j < JG; ++j) x[j][i] = read_x(buf, i, 4 * (p * JG + j) + g);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int at = (p * NB + b) & 1;
          s[at] = scales_of<SF16>(lds_read(reinterpret_cast<const u32x2*>(
              s_x[buf] + kScAt + wave * kScWave + ((b * GPT + p) * 16 + 4 * g) * 2)));
#pragma unroll
          for (int j = 0; j < JG; ++j) {
            const u32x4 w = int_codes(q.w[0][b][p * JG + j], bits, X());
#pragma unroll
            for (int i = 0; i < MT; ++i) sum[at][i] = mfma(w, x[j][i], j ? sum[at][i] : first[i], X());
          }
          if (p + b > 0) scale_in(at ^ 1, (b + NB - 1) % NB);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      scale_in((GPT * NB - 1) & 1, NB - 1);
    }
  };

  // One barrier per step: past it the step's rows have landed for every wave (each waited for its own loads)
  // and every wave is done with the step before, whose buffer the next loads overwrite.
  Codes q[2];
  load_x(step0, 0);
  load_w(q[0], step0);
  for (int st = step0; st < step1; st += 2) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      if (st + d >= step1) break;
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      if (st + d + 1 < step1) {
        load_x(st + d + 1, d ^ 1);
        load_w(q[d ^ 1], st + d + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      compute(q[d], d);
      // The step's sums end here: put off behind the next loads, they would take registers that there are not.
#ifdef __HIP_DEVICE_COMPILE__  // the host has no such registers
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) asm volatile("" : "+v"(acc[i][b]));
#endif
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  if constexpr (kMx && __is_same(X, __bf16)) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (__any(top[b] > 252)) {  // the same way for the whole wave
#pragma unroll
        for (int i = 0; i < MT; ++i) mx_back4(acc[i][b], top[b]);
      }
  }
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    const int n = (nt0 + b) * 16 + 4 * g;
    if (n >= a.n) continue;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int row = m0 + 16 * i + c;
      if (row >= a.rows) continue;
      f32x4 y[MATS];
#pragma unroll
      for (int z = 0; z < MATS; ++z) {
        y[z] = acc[i][z * NT + b];
        if constexpr (kMx && __is_same(X, _Float16)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[z][e] = mx_back(y[z][e], a.top[z][n + e], X());
        }
      }
      if (m.parts > 1) {
#pragma unroll
        for (int z = 0; z < MATS; ++z)
          *reinterpret_cast<f32x4*>(m.part + (((int64_t)part * MATS + z) * a.rows + row) * m.npad + n) = y[z];
      } else {
        store4<MATS>(a, row, n, y[0], y[MATS - 1]);
      }
    }
  }
}

template <typename X, int GPT, bool SF16, int MATS>
void launch_many_scales(const ManyArgs& m, const ManyPlan& p, hipStream_t stream) {
  const auto go = [&](auto kernel) {
    PSISPEC_LAUNCH(MATS == 2 ? "w4_gated" : "w4_linear", kernel, dim3((unsigned)p.mblocks * p.nblocks * p.parts),
                   dim3(256), 0, stream, m);
  };
  if (p.nb == 4)
    go((k_w4_many<X, GPT, MATS, SF16, 4>));
  else
    go((k_w4_many<X, GPT, MATS, SF16, 2>));
}

template <typename X, int GPT, int MATS>
hipError_t launch_many(const W4Args& a, hipStream_t stream) {
  constexpr bool kF8 = __is_same(X, F8);
  const ManyPlan p = many_plan(a.rows, a.n, a.k, MATS, GPT > 0 ? PSISPEC_W4_INT : PSISPEC_W4_MX);
  ManyArgs m{a, static_cast<float*>(a.workspace), nullptr, p.mpad, p.npad, p.mblocks, p.nblocks, p.parts, kF8 ? p.steps / 2 : p.steps, p.band};
  m.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + p.part_at);
  if constexpr (!kF8 && GPT > 0) {
    const int64_t blocks = (int64_t)p.mpad / 16 * ((a.ktiles + kSumTiles - 1) / kSumTiles);  // a launch takes less than 2^32 threads
    PSISPEC_LAUNCH("w4_sums", (k_w4_sums<X>), dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), dim3(256), 0,
                   stream, m);
  }
  if (GPT > 0 && a.scale_f16)
    launch_many_scales<X, GPT, GPT != 0, MATS>(m, p, stream);
  else
    launch_many_scales<X, GPT, false, MATS>(m, p, stream);
  if (p.parts > 1) {
    const int64_t all = (int64_t)a.rows * p.npad / 4;
    PSISPEC_LAUNCH("w4_join", k_w4_join<MATS>, dim3((unsigned)((all + 255) / 256)), dim3(256), 0, stream, m);
  }
  return hipGetLastError();
}

}  // namespace w4
}  // namespace psispec
