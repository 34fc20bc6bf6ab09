// attend.h -- the attention kernel over the paged cache (one instantiation set per translation unit).
//
//   out_m = sum_t w_mt v_t / sum_t w_mt,  w_mt = exp2(x_mt - max), x_mt = scale log2(e) q_m . k_t
//
// One key/value head serves G query heads, so its query rows (block row i, head g) -> m = i G + g share
// every key and value read: they form the 16-row tiles of the matrix products.  A workgroup's job is
// (line, key/value head, group of up to 16 MT rows), and its four waves take disjoint runs of
// 32-position tiles, each with softmax statistics of its own, that are joined at the end.  With heads in
// fours a job is four heads, so that neighbouring heads of the same positions are read at about the
// same time (one after the other, the 128- and 256-byte pieces of a position cost HBM about a tenth of
// its rate): with few rows each wave has one of them to itself and joins nothing, with many (whose
// queries are in LDS) each of four workgroups of an XCD has one.
//
// Products (v_mfma_f32_16x16x32, 32-bit sums).  Transposed, so that a lane owns one query row:
//   S^T = K Q^T   A = 16 positions x 32 dims of K, B = Q (in registers for the whole job)
//   O^T = V^T P^T A = 16 dims x 32 positions of V (transposing LDS reads), B = P
// The lane (row l % 16, group g = l / 16) that gets scores of positions 4g..4g+3 of both 16-position
// halves holds exactly the B fragment of the second product when its contraction index (g, j) is
// read as position 16 (j / 4) + 4 g + j % 4: weights go from one product to the next in registers.
// The running maximum and sum are per lane; the maximum is raised (and sums rescaled) only when a score
// exceeds it by more than 2^8, so most tiles need no exchange between lanes.  P is split into a
// 16-bit pair (hi + lo, relative error 2^-16) and multiplied twice: a single 16-bit P would add an
// error as large as the output's own rounding, and the product is not what bounds the kernel.
// The pair is of bf16, whose range is that of 32 bits (8-bit V widens to either type exactly), but for
// f16 V: f16 ends at 2^-24, and weights below 2^-9 would lose bits of the pair, those below 2^-25 all,
// while the sum l keeps them (a position far above the others with a value of 0 shows it).  There the
// weights are taken times 2^14 and relative to a reference that follows the tiles down too: it is
// raised by scores 2^1 above it and lowered when a tile has nothing within 2^8 of it, at most by 2^64
// (what lies deeper is below f16's range).  A weight is then off by 2^-16 of itself or
// 2^-39 of the reference's; over all positions at most 2^-26 of the largest |v|.  Cost, f16 caches
// alone (the measured lines below): 64 lines of one row 185.8 -> 186.8 us, of 9 rows 118.7 -> 121.8, trees 68.9 ->
// 69.7.
//
// Memory.  K and V go from HBM to LDS by 16-byte direct loads (no registers), each wave into a
// ring of its own (no barrier in the loop): K and V of a tile have separate places, each refilled as
// soon as its product is done, so one of the two is always in flight.  A row's 16-byte chunks are
// permuted by its position (on the load's source side) so that the reads of 16 rows at one chunk
// meet no LDS bank twice.  Page ids come 64 at a time, one in each lane.
//
// Work.  All jobs of the call laid end to end, in steps of 128 positions, are cut into one share per
// workgroup, however uneven the lines are; a job cut by a border leaves its parts (maximum, sum,
// unnormalised output in 32 bits) in the workspace and k_attend_join adds them in order.
//
// Measured, 32 query and 8 key/value heads of 128 (the kernel, then the join): 64 lines of 1000-8000
// positions, one row each, 186 us (6.3 TB/s of keys and values) + 5.3; 64 lines of 300-4200, 9 rows, 121
// (4.7 TB/s; three idle and every fifth with 5 rows, all with 9: 128, the same rate) + 7; 8 lines of 3500-4500, trees of 33 rows, 71 + 6; 4 lines of 125 000 in 8 bits 163 (6.3
// TB/s) + 7; one line of 500, 9.5 + 5.2.  The loads alone take 184 and 118 of the first two, the products
// and softmax alone 48 and 74.  HBM bounds one row (from L2 the same kernel reads 10-11 TB/s); with three
// row tiles a tile's own time bounds the waves (5.8 TB/s at most, from L2 as well), then the ends of
// jobs (pipeline refilled, waves joined, about 4 us each).
#pragma once

#include <type_traits>

#include "paged.h"

namespace psispec {

constexpr int kAttendCUs = 256;
constexpr int kAttendWaves = 4;
constexpr int kAttendThreads = 64 * kAttendWaves;
constexpr int kAttendTile = 32;                          // positions per tile
// Cache policy of the tiles: nontemporal when each is read once (64 lines of 1000-8000 positions:
// 210 us without, 187 with); kept when several row groups of a job read them (33-row trees: 89 us
// nontemporal, 79 kept).  The path for heads and pages of any size is nontemporal throughout (not
// measured kept).
constexpr int kNonTemporal = 2;

// The shares: one per workgroup that runs at once (R of them), or one per unit of work if there are
// fewer.  A unit is a step, and every job has `job_cost` units more at its start for what a job costs
// beside its steps.  Workgroups are dealt to the 8 XCDs in turn; each XCD gets a contiguous run of
// shares, so that the row groups and heads that read the same pages meet in one L2.  Of the two
// workgroups on a CU the one launched later is slower by a seventh, so the shares of the first half
// of an XCD's workgroups are larger (34 : 30; 64 lines of 9 rows 120.0 us, even shares 122.7), except
// below two units a share, where the small ones could be empty: a job's parts lie in shares one behind
// the other.  More, smaller shares given out as places become free even out the rest, and lose more than
// that to joining.
constexpr int kXcds = 8;
__host__ __device__ inline int64_t share_start(int64_t all, int64_t shares, int R, int skew, int64_t w) {
  if (shares < R) return w;
  const int64_t per = R / kXcds, h = per / 2, first = all >= 2 * R ? 32 + skew : 32;
  const int64_t x = w / per, j = w - x * per;
  const int64_t at = j < h ? first * j : first * h + (64 - first) * (j - h);
  return all * (x * 64 * h + at) / (kXcds * 64 * h);
}
// the share that holds a unit
__host__ __device__ inline int64_t share_of(int64_t all, int64_t shares, int R, int skew, int64_t unit) {
  int64_t lo = 0, hi = shares;  // start(lo) <= unit < start(hi)
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (share_start(all, shares, R, skew, mid) <= unit)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// A job that starts in share w and ends in a later one (parts == 0: none); h: head group.  One per job
// that has a step, or, with more jobs than shares, one per share.
struct AttendInfo {
  int32_t r, h, mt, parts, slot, w, pad[2];
};

struct AttendPlan {
  int mt;         // 16-row tiles per job
  int nmt;        // groups of 16 mt rows per (line, head)
  int dp;         // head dimension rounded up to 64, 128 or 256
  int wgs;        // workgroups
  int sub;        // workgroups per share
  int mask_words; // 64-bit words of a block row's mask (tree)
  int hpj;        // heads per job
  int prow;       // rows of a part in the workspace: the job's, at most blk G rounded up to 4
  size_t off_ml, off_o, off_mask, total;
};

struct AttendKernelArgs {
  AttendArgs a;
  int G, nmt, mask_words;
  int shares, skew;          // shares of a full grid; 2: an XCD's first half of them is larger
  int used;                  // shares of this grid, the others have no unit
  int solo;                  // a job per wave, whole jobs only (not with the queries in LDS)
  int step_tiles;            // tiles of each wave in a step
  int job_cost;              // units of a job beside its steps
  int hpj, hgroups;          // heads per job (1 or 4), groups of them
  int prow;                  // rows of a part in the workspace
  uint32_t ps_magic;         // ceil(2^32 / page_size)
  int halves;                // whole heads of DP dims, pages of 16-position multiples, strides below 2^31
  uint32_t page_bytes, row_bytes;  // the strides in bytes when halves
  float c;                   // scale log2(e)
  int by_job;                // info per job
  AttendInfo* info;          // [jobs or shares]
  float2* ml;                // [2 shares][hpj][prow]
  float* o;                  // [2 shares][hpj][prow][DP]
  const uint64_t* mask;      // [batch][blk][mask_words] or null
};

// rows of a job that are live and the positions that it reads
__device__ __host__ inline int job_keys(int L, int n, int G, int mt, int rows) {
  const int first = mt * rows / G;
  if (first >= n) return 0;
  int last = (mt * rows + rows - 1) / G;
  if (last > n - 1) last = n - 1;
  return L + last + 1;
}

// Two workgroups per CU (64 KiB rings, 256 registers per lane) for heads up to 128, one (128 KiB, 512
// registers) beyond.
__host__ __device__ constexpr bool attend_two(int dp) { return dp <= 128; }

// With many rows the queries' fragments stay in LDS instead of registers.
__host__ __device__ constexpr bool attend_q_lds(int dp, int mt) { return mt * dp > 256 || mt >= 4; }

// Launchers, one per translation unit
hipError_t launch_attend_bf16(const AttendKernelArgs& k, int dp, int mt, hipStream_t stream);
hipError_t launch_attend_f16(const AttendKernelArgs& k, int dp, int mt, hipStream_t stream);
hipError_t launch_attend_bf16_f8(const AttendKernelArgs& k, int dp, int mt, hipStream_t stream);
hipError_t launch_attend_f16_f8(const AttendKernelArgs& k, int dp, int mt, hipStream_t stream);

namespace attend {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_void;

template <typename T> struct Elem;
template <> struct Elem<__bf16> {
  typedef __bf16 x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 x4 __attribute__((ext_vector_type(4)));
  typedef __bf16 x8 __attribute__((ext_vector_type(8)));
  static constexpr uint32_t kExpStep = 0x00800080u;
  __device__ static f32x4 mfma(x8 a, x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  template <bool HI> __device__ static x2 from_f8(uint32_t w) {
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI);
  }
  __device__ static x4 tr(const __attribute__((address_space(3))) x4* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) x4*)p);
  }
};
template <> struct Elem<_Float16> {
  typedef _Float16 x2 __attribute__((ext_vector_type(2)));
  typedef _Float16 x4 __attribute__((ext_vector_type(4)));
  typedef _Float16 x8 __attribute__((ext_vector_type(8)));
  static constexpr uint32_t kExpStep = 0x04000400u;
  __device__ static f32x4 mfma(x8 a, x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  template <bool HI> __device__ static x2 from_f8(uint32_t w) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI);
  }
  __device__ static x4 tr(const __attribute__((address_space(3))) x4* p) {
    typedef short i16x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                      (__attribute__((address_space(3))) i16x4*)p));
  }
};

// LDS reads.  The restrict-qualified (inlined) parameters give the accesses alias scopes of their
// own, so the compiler adds no wait for the direct-to-LDS loads in flight: the kernel orders those
// itself (vmcnt waits before a tile is read, a wait for its reads before it is refilled).
template <typename V>
__device__ __attribute__((always_inline)) inline V lds_read(const char* __restrict__ p) {
  return *reinterpret_cast<const V*>(p);
}
template <typename T>
__device__ __attribute__((always_inline)) inline typename Elem<T>::x4 lds_tr16(
    const char* __restrict__ p) {
  typedef typename Elem<T>::x4 x4;
  return Elem<T>::tr((const __attribute__((address_space(3))) x4*)p);
}
__device__ __attribute__((always_inline)) inline i32x2 lds_tr8(const char* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)p);
}

// 16 bytes per lane straight to LDS, lane l's at to + 16 l (to: wave-uniform)
template <int POLICY> __device__ inline void load_lds(const char* from, char* to) {
  __builtin_amdgcn_global_load_lds((global_void*)from, (lds_void*)to, 16, 0, POLICY);
}

// eight 8-bit numbers as T (exact)
template <typename T>
__device__ inline typename Elem<T>::x8 widen(uint32_t w0, uint32_t w1) {
  typedef Elem<T> E;
  typename E::x8 y;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const typename E::x2 lo = E::template from_f8<false>(e ? w1 : w0);
    const typename E::x2 hi = E::template from_f8<true>(e ? w1 : w0);
    y[4 * e] = lo[0];
    y[4 * e + 1] = lo[1];
    y[4 * e + 2] = hi[0];
    y[4 * e + 3] = hi[1];
  }
  return y;
}

// all ones in the places of a word's finite elements, zeros in those of NaN and infinities
template <typename T, bool F8> __device__ inline uint32_t finite_mask(uint32_t w) {
  // adding one step of the exponent (8 bits: of the whole number) carries out of all ones
  if constexpr (F8) {
    const uint32_t m = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    return ~((m >> 7) * 0xffu);
  } else {
    const uint32_t m = ((w & 0x7fff7fffu) + Elem<T>::kExpStep) & 0x80008000u;
    return ~((m >> 15) * 0xffffu);
  }
}

// Wait until at most units * UNIT loads are outstanding (units wave-uniform, at most MAX).
template <int N> __device__ inline void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N > 63 ? 63 : N) : "memory");
}
template <int UNIT, int MAX> __device__ inline void wait_vm(int units) {
  if constexpr (MAX == 0) {
    wait_loads<0>();
  } else {
    if (units >= MAX)
      wait_loads<MAX * UNIT>();
    else
      wait_vm<UNIT, MAX - 1>(units);
  }
}
// Wait for the results of the matrix instructions before this point.  The hardware does not hold a
// reader back, and the waits that the compiler puts in do not always reach across the branch that
// follows here: a reader on its taken side got a sum without its last product.
__device__ inline void wait_matrix() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ inline void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Maximum / sum over the four 16-lane groups of a wave (lanes l, l^16, l^32, l^48).
__device__ inline float group_max(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ inline float group_sum(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Exclusive sum over the workgroup; *total: the whole.  s: one int64 of LDS per wave.
__device__ inline int64_t block_scan(int64_t x, int64_t* s, int64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t inc = x;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t y = __shfl_up(inc, o, 64);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 63) s[wave] = inc;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kAttendWaves; ++w) {
    before += w < wave ? s[w] : 0;
    all += s[w];
  }
  *total = all;
  return before + inc - x;
}

// steps of job group mt of a line: a step is step_tiles tiles of each wave
template <bool Q_LDS> __device__ inline int job_steps(const AttendKernelArgs& k, int keys) {
  const int step = kAttendTile * (Q_LDS ? kAttendWaves : kAttendWaves / k.hpj) * k.step_tiles;
  return (keys + step - 1) / step;
}
template <bool Q_LDS>
__device__ inline int64_t line_units(const AttendKernelArgs& k, int r, int rows) {
  int L, n;
  if (!line_rows(k.a.len, k.a.n_new, r, k.a.blk, k.a.c.slots, k.a.c.page_size, &L, &n) || n == 0)
    return 0;
  int64_t s = 0;
  for (int mt = 0; mt < k.nmt; ++mt) {
    const int keys = job_keys(L, n, k.G, mt, rows);
    s += keys > 0 ? job_steps<Q_LDS>(k, keys) + k.job_cost : 0;
  }
  return s * k.hgroups;
}

// A workgroup's LDS: the waves' rings of K and V tiles, and for many rows the queries.
template <int RB, int MT, int DP> struct Shape {
  static constexpr bool kTwo = attend_two(DP);
  static constexpr int kStage = 2 * kAttendTile * RB;  // K and V of one tile
  static constexpr int kRing = (kTwo ? 65536 : 131072) / kAttendWaves;
  static constexpr int kStages = kRing / kStage;
  static constexpr int kPerCU = kTwo ? 2 : 1;
  static constexpr bool kQLds = attend_q_lds(DP, MT);
  static constexpr int kLds = kRing * kAttendWaves + (kQLds ? MT * 16 * DP * 2 : 0);
};

// Where chunk c of row `row` lies in the row: at c ^ swz(row).  Both are bitwise in the row (so
// swz(a + b) = swz(a) ^ swz(b) for disjoint bits), and chosen so that the lanes of one read spread over
// all banks: a K read takes one chunk of 16 rows, a 16-bit V read two neighbouring chunks of 8 rows
// per half wave, an 8-bit V read one chunk of 16 rows (0-7 and 16-23) per half wave.
template <int RB> __device__ __host__ constexpr int swz_k(int row) {
  return (row / (RB >= 256 ? 1 : 256 / RB)) & ((RB >= 256 ? 16 : RB / 16) - 1);
}
template <int RB, bool F8> __device__ __host__ constexpr int swz_v(int row) {
  return F8 ? (((row & 7) | ((row >> 4) & 1) << 3) / (RB >= 256 ? 1 : 256 / RB)) &
                  ((RB >= 256 ? 16 : RB / 16) - 1)
            : ((row / (RB >= 256 ? 1 : 256 / RB)) & ((RB >= 256 ? 16 : RB / 16) / 2 - 1)) << 1;
}

template <typename T, bool F8, int DP, int MT>
__global__ __launch_bounds__(kAttendThreads, (Shape<(F8 ? 1 : 2) * DP, MT, DP>::kPerCU))
void k_attend(AttendKernelArgs k) {
  typedef Elem<T> E;
  typedef typename E::x4 x4;
  typedef typename E::x8 x8;
  // the second product's type and its weights (see above)
  typedef typename std::conditional<F8, __bf16, T>::type P;
  typedef typename Elem<P>::x2 p2;
  typedef typename Elem<P>::x8 p8;
  constexpr bool kFollow = std::is_same<P, _Float16>::value;
  constexpr float kSlack = kFollow ? 1.0f : 8.0f;   // powers of two that a weight may exceed 1 by
  constexpr float kBias = kFollow ? 14.0f : 0.0f;   // the reference lies 2^kBias below (weights up to 2^15)
  constexpr float kDrop = 8.0f, kDeepest = 64.0f;
  constexpr int ES = F8 ? 1 : 2;
  constexpr int RB = DP * ES;                 // bytes of a row in LDS
  typedef Shape<RB, MT, DP> Sh;
  constexpr int NST = Sh::kStages;
  constexpr int CPR = RB / 16;                // 16-byte chunks of a row
  constexpr int RPI = 1024 / RB;              // rows that one load instruction fills
  constexpr int TILE = kAttendTile * RB;
  constexpr int NLD = TILE / 1024;            // load instructions per tile of K or V
  constexpr int ROWS = 16 * MT;
  constexpr int NT = DP / 16;                 // 16-dim tiles of the output
  constexpr int KS = DP / 32;                 // contraction steps of the first product
  static_assert(NST >= 1 && 4 * NST * NLD * 2 * 1024 <= 131072, "the ring fits the LDS");
  static_assert(16 * (DP + 4) * 4 <= Sh::kRing, "a wave's part of the output fits its ring");

  constexpr bool kQLds = Sh::kQLds;
  extern __shared__ __align__(1024) char ring[];  // [waves][stages][K tile, V tile], then queries
  char* const q_lds = ring + Sh::kRing * kAttendWaves;
  __shared__ float s_m[kAttendWaves][ROWS], s_l[kAttendWaves][ROWS];
  __shared__ int64_t s_scan[kAttendWaves];
  __shared__ int64_t s_base;
  __shared__ int s_line;

  const AttendArgs& a = k.a;
  const psispec_paged_cache& c = a.c;
  const int G = k.G, dim = c.dim;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  const int ps = c.page_size;

  // ---- this workgroup's share [x, x_end) of all units, and the line that holds unit x
  // units of the lines before line `tid`, of the line, and of all lines; the first 256 lines
  const int64_t mine0 = tid < a.batch ? line_units<kQLds>(k, tid, ROWS) : 0;
  int64_t all;
  const int64_t at0 = block_scan(mine0, s_scan, &all);
  int64_t base = all;
  if (a.batch > kAttendThreads) {
    int64_t more = 0, sum;
    for (int r0 = kAttendThreads; r0 < a.batch; r0 += kAttendThreads)
      more += r0 + tid < a.batch ? line_units<kQLds>(k, r0 + tid, ROWS) : 0;
    block_scan(more, s_scan, &sum);
    all += sum;
  }
  const int64_t shares = min(all, (int64_t)k.shares);
  const int nsub = kQLds ? k.hpj : 1;
  const int nth = shares < k.shares ? blockIdx.x : blockIdx.x % kXcds * (gridDim.x / kXcds) + blockIdx.x / kXcds;
  const int w = nth / nsub, sub = nth - w * nsub;
  if (tid == 0 && sub == 0 && !k.by_job) k.info[w].parts = 0;
  if (w >= shares) return;
  int64_t x = share_start(all, shares, k.shares, k.skew, w);
  const int64_t x0 = x, x_end = share_start(all, shares, k.shares, k.skew, w + 1);
  if (at0 <= x && x < at0 + mine0) {
    s_line = tid;
    s_base = at0;
  }
  for (int r0 = kAttendThreads; base <= x && r0 < a.batch; r0 += kAttendThreads) {
    const int64_t mine = r0 + tid < a.batch ? line_units<kQLds>(k, r0 + tid, ROWS) : 0;
    int64_t part;
    const int64_t at = base + block_scan(mine, s_scan, &part);
    if (at <= x && x < at + mine) {
      s_line = r0 + tid;
      s_base = at;
    }
    base += part;
  }
  __syncthreads();
  int r = s_line;
  int64_t off = x - s_base;  // unit within the line's jobs
  const bool solo = !kQLds && k.solo;

  char* const my_ring = ring + wave * Sh::kRing;
  bool first_segment = true;

  for (; r < a.batch; ++r) {  // lines of the share
    int L, n;
    const bool live_line =
        line_rows(a.len, a.n_new, r, a.blk, c.slots, ps, &L, &n) && n > 0;
    if (!live_line) continue;
    const int32_t* const tab = c.table + (int64_t)r * c.table_stride;
    for (int hg = 0; hg < k.hgroups && x < x_end; ++hg) {
      const int h = hg * k.hpj + (kQLds ? sub : k.hpj == 1 ? 0 : wave);
      for (int mt0 = 0; mt0 < k.nmt && x < x_end; ++mt0) {
        const int keys = job_keys(L, n, G, mt0, ROWS);
        const int steps = job_steps<kQLds>(k, keys);
        const int units = keys > 0 ? steps + k.job_cost : 0;
        if (off >= units) {
          off -= units;
          continue;
        }
        // ---- segment: units [off, off + take) of the job, its steps [step0, step1)
        const int64_t job_x = x - off;
        const int take = (int)min((int64_t)units - off, x_end - x);
        const int step0 = max((int)off - k.job_cost, 0);
        const int step1 = max((int)off + take - k.job_cost, 0);
        // solo: a job is one unit, and the waves take the share's in turn, so that neighbours in time are
        // neighbouring heads and row groups of the same positions
        const bool skip = step0 >= step1 || (solo && (int)(x - x0) % kAttendWaves != wave);
        x += take;
        off = 0;
        if (skip) continue;
        const int ntiles = (keys + kAttendTile - 1) / kAttendTile;
        const bool alone = solo || (!kQLds && k.hpj > 1);  // the wave has the head to itself
        const int splits = alone ? 1 : kAttendWaves;
        const int tile0 = step0 * splits * k.step_tiles;
        const int tile1 = min(step1 * splits * k.step_tiles, ntiles);
        const int cnt = tile1 - tile0;
        const int t0 = alone ? tile0 : tile0 + cnt * wave / kAttendWaves;
        const int t1 = alone ? tile1 : tile0 + cnt * (wave + 1) / kAttendWaves;

        // ---- loads: tile t into stage t % NST
        const int chunks = dim * ES / 16;       // real chunks of a row
        const int64_t head_off = (int64_t)h * c.head_stride * ES;
        const char* const kbase = static_cast<const char*>(c.k) + head_off;
        const char* const vbase = static_cast<const char*>(c.v) + head_off;
        int tab_chunk, tab_now = 0, tab_next, chunk_end = 0;
        const uint32_t lane_ofs = (uint32_t)(lane / CPR) * k.row_bytes;
        const int last_slot = (keys - 1) / ps;
        auto fetch_tab = [&](int chunk) { return tab[min(chunk * 64 + lane, last_slot)]; };
        {  // the first page ids are on their way while the queries are asked for
          tab_chunk = (int)((uint32_t)(t0 * kAttendTile) / (64u * ps)) - 1;
          tab_next = fetch_tab(tab_chunk + 1);
        }
        // tile t into `to`: row i * RPI + lane / CPR of each load instruction; rows behind the job's
        // last position are read as the last
        auto issue = [&](int t, const char* from, char* to, auto is_v) {
          const int tile_pos = t * kAttendTile;
          if (tile_pos >= chunk_end) {  // tiles never straddle 64 pages
            const int chunk = (uint32_t)tile_pos / (64u * ps);
            const int raw = chunk == tab_chunk + 1 ? tab_next : fetch_tab(chunk);
            tab_now = (uint32_t)raw < (uint32_t)c.num_pages ? raw : 0;  // a bad id stays in bounds
            tab_chunk = chunk;
            chunk_end = (chunk + 1) * 64 * ps;
            tab_next = fetch_tab(chunk + 1);
          }
          const int rel0 = tile_pos + 64 * ps - chunk_end;
          const int lane_row = lane / CPR;
          const int swz = is_v() ? swz_v<RB, F8>(lane_row) : swz_k<RB>(lane_row);
          const int lane_chunk = (lane % CPR) ^ swz;
          if (k.halves) {
            // each 16 positions of the tile lie in one page: two scalar addresses
            const int lim = keys - 1 + 64 * ps - chunk_end;
            const bool part = tile_pos + kAttendTile > keys;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t rel = min(rel0 + 16 * half, lim);
              const uint32_t idx = __umulhi(rel, k.ps_magic);
              const uint32_t page = (uint32_t)__builtin_amdgcn_readlane(tab_now, idx);
              const char* const at0 =
                  from + (uint64_t)page * k.page_bytes + (rel - idx * ps) * k.row_bytes;
              auto rows = [&](auto policy, auto is_part) {
                const char* at = at0;
#pragma unroll
                for (int i = half * NLD / 2; i < (half + 1) * NLD / 2; ++i) {
                  const int ch = lane_chunk ^ (is_v() ? swz_v<RB, F8>(i * RPI) : swz_k<RB>(i * RPI));
                  if constexpr (decltype(is_part)::value) {
                    const int row = min((i - half * NLD / 2) * RPI + lane_row, lim - (int)rel);
                    load_lds<decltype(policy)::value>(at0 + ((uint32_t)row * k.row_bytes + (ch << 4)),
                                                      to + i * 1024);
                  } else {
                    load_lds<decltype(policy)::value>(at + (lane_ofs + (ch << 4)), to + i * 1024);
                    at += RPI * k.row_bytes;
                  }
                }
              };
              if (part)
                rows(std::integral_constant<int, 0>{}, std::true_type{});
              else if (k.nmt > 1)
                rows(std::integral_constant<int, 0>{}, std::false_type{});
              else
                rows(std::integral_constant<int, kNonTemporal>{}, std::false_type{});
            }
          } else {
            const int lim = keys - 1 + 64 * ps - chunk_end;
#pragma unroll 2
            for (int i = 0; i < NLD; ++i) {
              const int rel = min(rel0 + i * RPI + lane_row, lim);
              const int idx = ps == 1 ? rel : (int)__umulhi((uint32_t)rel, k.ps_magic);
              const int page = __shfl(tab_now, idx, 64);
              const int ch = lane_chunk ^ (is_v() ? swz_v<RB, F8>(i * RPI) : swz_k<RB>(i * RPI));
              const char* const at =
                  from + ((int64_t)page * c.page_stride + (int64_t)(rel - idx * ps) * c.row_stride) * ES +
                  (ch << 4);
              if (ch < chunks)
                load_lds<kNonTemporal>(at, to + i * 1024);
            }
          }
        };
        const float sc_signed = k.c * (F8 && c.k_scale ? c.k_scale[h] : 1.0f);
        const float sc = fabsf(sc_signed);
        // ---- queries: row n16 of each 16-row tile, in registers, or for many rows in LDS in the
        // order of the fragments
        x8 qf[kQLds ? 1 : MT][kQLds ? 1 : KS], zq[kQLds ? MT * KS / kAttendWaves : 1];
        int irow[MT];  // block row, or -1 behind the job's last
        auto load_q = [&](int mt, int s) {
          const int m = mt0 * ROWS + mt * 16 + n16, i = m / G;
          const T* q = static_cast<const T*>(k.a.q) +
                       ((int64_t)r * k.a.blk + (i < n ? i : 0)) * k.a.q_stride +
                       (int64_t)(h * G + (m - i * G)) * dim;
          // the dims of the lane's K fragment: 16-bit rows, chunk 4 s + g; 8-bit rows, half s % 2 of
          // chunk 4 (s / 2) + g
          const int d = F8 ? (4 * (s >> 1) + g) * 16 + (s & 1) * 8 : (4 * s + g) * 8;
          x8 z = {};
          if (d < dim && i < n) z = *reinterpret_cast<const x8*>(q + d);
          return z;
        };
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int i = (mt0 * ROWS + mt * 16 + n16) / G;
          irow[mt] = i < n ? i : -1;
          if constexpr (!kQLds) {
#pragma unroll
            for (int s = 0; s < KS; ++s) qf[mt][s] = load_q(mt, s);
          }
        }
        if constexpr (kQLds) {
#pragma unroll
          for (int f = 0; f < MT * KS / kAttendWaves; ++f) {
            const int u = f * kAttendWaves + wave;
            zq[f] = load_q(u / KS, u % KS);
          }
        }

        char* const stage0 = my_ring;
        if (dim != DP) {  // the chunks behind the head's last are never loaded
          for (int b = lane * 16; b < Sh::kRing; b += 1024)
            *reinterpret_cast<u32x4*>(my_ring + b) = u32x4{0, 0, 0, 0};
          wait_lds();
        }
#pragma unroll
        for (int s = 0; s < NST; ++s) {
          if (t0 + s < t1) {
            issue(t0 + s, kbase, stage0 + s * Sh::kStage, std::false_type{});
            issue(t0 + s, vbase, stage0 + s * Sh::kStage + TILE, std::true_type{});
          }
        }
        // the queries, asked for before the tiles: a wait for them inside the loop would also wait for the
        // tiles in flight there
        if constexpr (kQLds) {
#pragma unroll
          for (int f = 0; f < MT * KS / kAttendWaves; ++f)
            *reinterpret_cast<x8*>(q_lds + ((f * kAttendWaves + wave) * 64 + lane) * 16) =
                sc_signed < 0.0f ? -zq[f] : zq[f];
          __syncthreads();
        } else {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              if (sc_signed < 0.0f) qf[mt][s] = -qf[mt][s];
              asm volatile("" : "+v"(qf[mt][s]));
            }
        }

        f32x4 acc[MT][NT];
        float m_run[MT], l_run[MT], top[kFollow ? MT : 1];  // the reference, the sum; the highest reference
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          m_run[mt] = kNegBig;
          if constexpr (kFollow) top[mt] = kNegBig;
          l_run[mt] = 0.0f;
#pragma unroll
          for (int d = 0; d < NT; ++d) acc[mt][d] = f32x4{0, 0, 0, 0};
        }

        // Positions pos0 .. pos0 + 31 that block row i (-1: none) sees, as bits; some reach behind L.
        auto visible = [&](int i, int pos0) -> uint32_t {
          if (!k.mask) {
            const int cnt = max(min(L + i + 1 - pos0, 32), 0);
            return (uint32_t)((1ull << cnt) - 1);
          }
          const uint64_t* const words =
              k.mask + ((int64_t)r * k.a.blk + max(i, 0)) * k.mask_words;
          const int j0 = pos0 - L, before = max(-j0, 0), j = max(j0, 0), sh = j & 63;
          const int w0 = min(j >> 6, k.mask_words - 1), w1 = min(w0 + 1, k.mask_words - 1);
          uint64_t bits = words[w0] >> sh;
          bits |= w1 > w0 && sh > 0 ? words[w1] << (64 - sh) : 0;
          return (uint32_t)((i < 0 ? 0 : bits) << before | ((1ull << before) - 1));
        };

        // ---- one tile; TAIL: it reaches behind the line's first L positions
        int st = 0;
        bool odd = false;
        auto tile = [&](int t, auto is_tail) {
          constexpr bool TAIL = decltype(is_tail)::value;
          char* const kt = stage0 + st * Sh::kStage;
          char* const vt = kt + TILE;
          // whole tiles in flight behind this one
          const int later = NST == 1 ? 0 : min(NST - 1, t1 - 1 - t);
          const bool refill = t + NST < t1;
          wait_vm<NLD, 2 * NST - 1>(1 + 2 * later);

          // ---- S^T = K Q^T
          f32x4 s[MT][2];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) s[mt][0] = s[mt][1] = f32x4{0, 0, 0, 0};
          const int k_at = n16 * RB + ((g ^ swz_k<RB>(n16)) << 4);
          u32x4 raw[2];
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            x8 kf[2];
            if constexpr (!F8) {
#pragma unroll
              for (int sub = 0; sub < 2; ++sub)
                kf[sub] = lds_read<x8>(kt + (k_at ^ (ks << 6)) + sub * 16 * RB);
            } else {
#pragma unroll
              for (int sub = 0; sub < 2; ++sub) {
                if (ks % 2 == 0) raw[sub] = lds_read<u32x4>(kt + (k_at ^ (ks / 2 << 6)) + sub * 16 * RB);
                kf[sub] = widen<T>(raw[sub][2 * (ks & 1)], raw[sub][2 * (ks & 1) + 1]);
              }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              x8 q;
              if constexpr (kQLds)
                q = lds_read<x8>(q_lds + ((mt * KS + ks) * 64 + lane) * 16);
              else
                q = qf[mt][ks];
              s[mt][0] = E::mfma(kf[0], q, s[mt][0]);
              s[mt][1] = E::mfma(kf[1], q, s[mt][1]);
            }
          }
          wait_lds();  // K is read: its place is free
          wait_matrix();
          if (refill) issue(t + NST, kbase, kt, std::false_type{});

          // ---- weights
          const int pos0 = t * kAttendTile;
          p8 p_hi[MT], p_lo[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t see = ~0u;
            if constexpr (TAIL) {
              see = visible(irow[mt], pos0) >> (4 * g);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                s[mt][e >> 2][e & 3] =
                    (see >> (16 * (e >> 2) + (e & 3))) & 1u ? s[mt][e >> 2][e & 3] : -INFINITY;
            }
            float mx = fmaxf(fmaxf(fmaxf(s[mt][0][0], s[mt][0][1]), fmaxf(s[mt][0][2], s[mt][0][3])),
                             fmaxf(fmaxf(s[mt][1][0], s[mt][1][1]), fmaxf(s[mt][1][2], s[mt][1][3])));
            // sc >= 0: a negative scale is in the queries' signs
            bool move;
            float m_new;
            if constexpr (kFollow) {
              // minus the largest exponent, rounded as the weight's own, so that no weight is too large
              const float x = fmaf(-mx, sc, m_run[mt]);
              // rows that see something here, and nothing near the reference
              uint64_t seen = __ballot(x < INFINITY), near = __ballot(x < kDrop - kBias);
              seen |= seen >> 32;
              near |= near >> 32;
              move = __any(x < -kBias - kSlack) || ((seen | seen >> 16) & ~(near | near >> 16) & 0xffffu) != 0;
            } else {
              mx *= sc;
              move = __any(mx > m_run[mt] + kSlack);
            }
            if (move) {
              mx = group_max(mx);
              if constexpr (kFollow) {
                const float g = mx * sc;
                m_new = g > -INFINITY ? fmaxf(g - kBias, top[mt] - kDeepest) : m_run[mt];
                // where 32 bits hold the reference in steps of 1 and more
                const float x = fmaf(-mx, sc, m_new);
                if (x < -kBias - kSlack) m_new += fmaxf(-x - kBias, fabsf(m_new) * 0x1p-23f);
                top[mt] = fmaxf(top[mt], m_new);
              } else {
                m_new = fmaxf(mx, m_run[mt]);
              }
              const float f = __builtin_amdgcn_exp2f(m_run[mt] - m_new);
              m_run[mt] = m_new;
              l_run[mt] *= f;
#pragma unroll
              for (int d = 0; d < NT; ++d) acc[mt][d] *= f;
            }
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              f32x2 p;
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                p[u] = __builtin_amdgcn_exp2f(fmaf(s[mt][(e + u) >> 2][(e + u) & 3], sc, -m_run[mt]));
                if constexpr (TAIL) p[u] = (see >> (16 * (e >> 2) + ((e + u) & 3))) & 1u ? p[u] : 0.0f;
              }
              sum += p[0] + p[1];
              const p2 hi = __builtin_convertvector(p, p2);
              const p2 lo = __builtin_convertvector(p - __builtin_convertvector(hi, f32x2), p2);
              p_hi[mt][e] = hi[0];
              p_hi[mt][e + 1] = hi[1];
              p_lo[mt][e] = lo[0];
              p_lo[mt][e + 1] = lo[1];
            }
            l_run[mt] += sum;
          }

          // ---- O^T += V^T P^T
          if (refill)
            wait_loads<(2 * NST - 1) * NLD>();
          else
            wait_vm<NLD, 2 * NST - 2>(2 * later);
          if constexpr (TAIL) {
            // Rows behind the job's last position hold a copy of it: zero them.  Block rows may hold
            // NaN or infinities that some of the queries do not see, and 0 * inf is not 0: such values
            // (rare) become 0 here and are added at the end, to the rows that see them.
#pragma unroll
            for (int i = 0; i < NLD; ++i) {
              if (pos0 + (i + 1) * RPI <= L) continue;
              char* const at = vt + i * 1024 + lane * 16;
              const int pos = pos0 + i * RPI + lane / CPR;
              u32x4 v = lds_read<u32x4>(at);
              uint32_t lost = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t keep = pos >= keys ? 0u : pos >= L ? finite_mask<T, F8>(v[e]) : ~0u;
                lost |= pos < keys ? ~keep : 0u;
                v[e] &= keep;
              }
              odd |= lost != 0;
              *reinterpret_cast<u32x4*>(at) = v;
            }
            wait_lds();
          }
#pragma unroll
          for (int d = 0; d < NT; ++d) {
            p8 vf;  // the lane's 8 positions of dims 16 d .. 16 d + 15
            if constexpr (!F8) {
              // group g, lane i of it: address of position 4 g + i / 4, dims 4 (i % 4) of the tile
              const int row = 4 * g + (n16 >> 2);
              const int v_at = row * RB + ((((n16 & 3) >> 1) ^ swz_v<RB, F8>(row)) << 4) + (n16 & 1) * 8;
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const x4 v4 = lds_tr16<T>(vt + (v_at ^ (d << 5)) + half * 16 * RB);
#pragma unroll
                for (int e = 0; e < 4; ++e) vf[4 * half + e] = v4[e];
              }
            } else {
              // lane i: position j = i / 2 of the group's eight, 8 of the 16 dims
              const int j = n16 >> 1;
              const int row = 16 * (j >> 2) + 4 * g + (j & 3);
              const int v_at = row * RB + (swz_v<RB, F8>(row) << 4) + (n16 & 1) * 8;
              const i32x2 v = lds_tr8(vt + (v_at ^ (d << 4)));
              vf = widen<P>((uint32_t)v[0], (uint32_t)v[1]);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              acc[mt][d] = Elem<P>::mfma(vf, p_hi[mt], acc[mt][d]);
              acc[mt][d] = Elem<P>::mfma(vf, p_lo[mt], acc[mt][d]);
            }
          }
          wait_lds();  // V is read: its place is free
          wait_matrix();
          if (refill) issue(t + NST, vbase, vt, std::true_type{});
          st = st + 1 == NST ? 0 : st + 1;
        };
        int t = t0;
        for (const int tm = min(t1, L / kAttendTile); t < tm; ++t) tile(t, std::false_type{});
        for (; t < t1; ++t) tile(t, std::true_type{});
        if constexpr (kFollow) {  // from here on relative to the highest reference
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if (!__any(m_run[mt] < top[mt])) continue;
            const float f = __builtin_amdgcn_exp2f(m_run[mt] - top[mt]);
            m_run[mt] = top[mt];
            l_run[mt] *= f;
#pragma unroll
            for (int d = 0; d < NT; ++d) acc[mt][d] *= f;
          }
        }

        // ---- the job's output, or its part
        const bool whole = step0 == 0 && step1 == steps;
        const int64_t slot = 2 * (int64_t)w + (first_segment ? 0 : 1);
        const float vscale = F8 && c.v_scale ? c.v_scale[h] : 1.0f;
        // dims d .. d+3 of row `row` of the job: the sums y over maximum m and weight l
        auto finish = [&](int row, int d, f32x4 y, float m, float l, bool any_odd) {
          const int q = mt0 * ROWS + row;
          const int i = q / G;
          if (any_odd) {  // NaN and infinities of the block rows that this row sees
            const int j1 = min(tile1 * kAttendTile, keys) - L;
            for (int j = max(tile0 * kAttendTile - L, 0); j < j1; ++j) {
              const bool on = (visible(i < n ? i : -1, L + j) & 1u) != 0;
              const int s = (L + j) / ps;
              const int page = (uint32_t)tab[s] < (uint32_t)c.num_pages ? tab[s] : 0;
              const char* v = static_cast<const char*>(c.v) + head_off + min(d, dim - 4) * ES +
                              ((int64_t)page * c.page_stride + (int64_t)(L + j - s * ps) * c.row_stride) * ES;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float z;
                if constexpr (F8)
                  z = (float)E::template from_f8<false>(reinterpret_cast<const uint8_t*>(v)[e])[0];
                else
                  z = (float)reinterpret_cast<const T*>(v)[e];
                y[e] += on && !__builtin_isfinite(z) ? z : 0.0f;
              }
            }
          }
          if (i >= n) return;
          if (whole) {
            if (d >= dim) return;
            const float f = vscale / l;
            x4 z;
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = (T)(y[e] * f);
            *reinterpret_cast<x4*>(static_cast<T*>(a.out) + ((int64_t)r * a.blk + i) * a.out_stride +
                                   (int64_t)(h * G + (q - i * G)) * dim + d) = z;
          } else {
            const int64_t at = (slot * k.hpj + (h - hg * k.hpj)) * k.prow + row;
            *reinterpret_cast<f32x4*>(k.o + at * DP + d) = y;
            if (d == 0) k.ml[at] = make_float2(m, l);
          }
        };
        if (alone) {
          const bool any_odd = __any(odd);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float l = group_sum(l_run[mt]);
#pragma unroll
            for (int d = 0; d < NT; ++d)
              finish(mt * 16 + n16, 16 * d + 4 * g, acc[mt][d], m_run[mt], l, any_odd);
          }
        } else {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float l = group_sum(l_run[mt]);
            if (g == 0) {
              s_m[wave][mt * 16 + n16] = m_run[mt];
              s_l[wave][mt * 16 + n16] = l;
            }
          }
          const bool any_odd = __syncthreads_or(odd);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float mx = kNegBig;
#pragma unroll
            for (int u = 0; u < kAttendWaves; ++u) mx = fmaxf(mx, s_m[u][mt * 16 + n16]);
            const float f = __builtin_amdgcn_exp2f(m_run[mt] - mx);
            char* const mine = my_ring + n16 * (DP + 4) * 4 + 4 * g * 4;
#pragma unroll
            for (int d = 0; d < NT; ++d)
              *reinterpret_cast<f32x4*>(mine + 16 * d * 4) = acc[mt][d] * f;
            __syncthreads();
            for (int it = tid; it < 16 * DP / 4; it += kAttendThreads) {
              const int row = it / (DP / 4), d = (it - row * (DP / 4)) * 4;
              f32x4 y = {0, 0, 0, 0};
              float rm = kNegBig, rl = 0.0f;
#pragma unroll
              for (int u = 0; u < kAttendWaves; ++u) {
                y += *reinterpret_cast<const f32x4*>(ring + u * Sh::kRing + row * (DP + 4) * 4 + d * 4);
                rm = fmaxf(rm, s_m[u][mt * 16 + row]);
              }
#pragma unroll
              for (int u = 0; u < kAttendWaves; ++u)
                rl += s_l[u][mt * 16 + row] * __builtin_amdgcn_exp2f(s_m[u][mt * 16 + row] - rm);
              finish(mt * 16 + row, d, y, rm, rl, any_odd);
            }
            __syncthreads();
          }
        }
        if (step0 == 0 && tid == 0 && sub == 0 && (!whole || k.by_job)) {  // the job starts here
          AttendInfo& o = k.info[k.by_job ? (r * k.hgroups + hg) * k.nmt + mt0 : w];
          o.r = r;
          o.h = hg;
          o.mt = mt0;
          o.slot = (int)slot;
          o.w = w;
          o.parts = whole ? 0 : (int)(share_of(all, shares, k.shares, k.skew, job_x + units - 1) - w) + 1;
        }
        first_segment = false;
      }
    }
    if (x >= x_end) return;
  }
}

template <typename T, bool F8, int DP, int MT>
hipError_t launch_one(const AttendKernelArgs& k, hipStream_t stream) {
  typedef Shape<(F8 ? 1 : 2) * DP, MT, DP> Sh;
  constexpr int shm = Sh::kLds;
  // more dynamic LDS than the default limit, once per device
  static unsigned long long done = 0;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev >= 64 || !(__atomic_load_n(&done, __ATOMIC_RELAXED) >> dev & 1)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_attend<T, F8, DP, MT>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, shm);
    if (e != hipSuccess) return e;
    if (dev < 64) __atomic_fetch_or(&done, 1ull << dev, __ATOMIC_RELAXED);
  }
  PSISPEC_LAUNCH("attend", (k_attend<T, F8, DP, MT>), dim3((unsigned)(k.used * (Sh::kQLds ? k.hpj : 1))),
                 dim3(kAttendThreads), shm, stream, k);
  return hipGetLastError();
}

template <typename T, bool F8>
hipError_t launch_typed(const AttendKernelArgs& k, int dp, int mt, hipStream_t stream) {
  if (dp == 64) {
    switch (mt) {
      case 1: return launch_one<T, F8, 64, 1>(k, stream);
      case 2: return launch_one<T, F8, 64, 2>(k, stream);
      case 4: return launch_one<T, F8, 64, 4>(k, stream);
    }
  } else if (dp == 128) {
    switch (mt) {
      case 1: return launch_one<T, F8, 128, 1>(k, stream);
      case 2: return launch_one<T, F8, 128, 2>(k, stream);
      case 3: return launch_one<T, F8, 128, 3>(k, stream);
    }
  } else if (dp == 256) {
    switch (mt) {
      case 1: return launch_one<T, F8, 256, 1>(k, stream);
      case 2: return launch_one<T, F8, 256, 2>(k, stream);
    }
  }
  return hipErrorInvalidValue;
}

}  // namespace attend
}  // namespace psispec
