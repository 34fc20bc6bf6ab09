// attend.hip -- attention over the paged cache: the shapes of its launches, the masks of a tree, and
// the join of the parts that the attention kernel's shares leave.
#include "attend.h"

namespace psispec {
namespace {

using attend::f32x4;

constexpr int kJoinRows = 4;

// Lines of tables up to this width (positions) are not cut: nothing is joined and the second launch goes.
// Kernels' time uncut against cut and joined: 9 rows of 8 heads 19.1 against 22.8 us at 250 positions, 21.5
// against 22.6 at 500, 25.0 against 22.8 at 750; 16 lines of one row 18.4 against 20.3 at 500.  One
// line of one row is cut sooner (heads in fours leave its waves alone with their positions): 14.0
// against 14.3 at 250, 16.3 against 15.1 at 500.
constexpr int64_t kWholePositions = 512, kWholeFewPositions = 256;
constexpr int kFewHeads = 64;
// Many of them (two per workgroup and more) take a wave each, in row tiles few enough for the queries in
// registers: no barriers, four jobs at once in a workgroup.  95 lines of 16 heads, 19 rows and 10
// positions 76 -> 46 us, 83 lines of one row 30 -> 23; 128 lines of 8 heads, one row of 450 positions 52 -> 48.
// Where that needs more row groups than the plan has, only up to kSoloPositions: 256 lines of 8 heads and 9
// rows 79 -> 58 us at 200 positions, but 110 -> 117 at 450.
constexpr int64_t kSoloPositions = 256;

// Row tiles of a job and jobs per (line, key/value head) for M = blk G query rows.  As few groups as
// the instantiated sizes allow (each group reads every key and value again), then the smallest
// size that holds a group: rows that pad a tile cost matrix work.  The largest sizes are those with
// which two workgroups run on a CU: 132 rows of 128 dims took 102 us as two groups of 5 tiles, one
// wave per SIMD, and 92 us as three groups of 3 although every position is read three times.
AttendPlan make_attend_plan(int batch, int blk, int heads_q, int heads_kv, int dim) {
  AttendPlan p{};
  p.dp = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
  static const int k64[] = {1, 2, 4}, k128[] = {1, 2, 3}, k256[] = {1, 2};
  const int* sizes = p.dp == 64 ? k64 : p.dp == 128 ? k128 : k256;
  const int ns = p.dp == 256 ? 2 : 3;
  const int64_t rows = (int64_t)blk * (heads_q / heads_kv);
  const int most = sizes[ns - 1] * 16;
  p.nmt = (int)((rows + most - 1) / most);
  const int tiles = (int)(((rows + p.nmt - 1) / p.nmt + 15) / 16);
  for (int i = ns - 1; i >= 0; --i)
    if (sizes[i] >= tiles) p.mt = sizes[i];
  p.nmt = (int)((rows + p.mt * 16 - 1) / (p.mt * 16));
  p.wgs = (attend_two(p.dp) ? 2 : 1) * kAttendCUs;
  p.mask_words = (blk + 63) / 64;
  p.hpj = heads_kv % 4 == 0 ? 4 : 1;
  p.sub = attend_q_lds(p.dp, p.mt) ? p.hpj : 1;
  p.prow = (int)((rows < p.mt * 16 ? rows : p.mt * 16) + kJoinRows - 1) / kJoinRows * kJoinRows;
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t at = off;
    off = (off + n + 255) / 256 * 256;
    return at;
  };
  take(sizeof(AttendInfo) * p.wgs);
  p.off_ml = take(sizeof(float2) * 2 * (p.wgs / p.sub) * p.hpj * p.prow);
  p.off_o = take(sizeof(float) * 2 * (p.wgs / p.sub) * p.hpj * p.prow * (size_t)p.dp);
  p.off_mask = take(sizeof(uint64_t) * (size_t)batch * blk * p.mask_words);
  p.total = off;
  return p;
}

// A tree's masks: row j's word w holds bit i for every ancestor-or-self 64 w + i of row j.
__global__ __launch_bounds__(256) void k_tree_mask(AttendArgs a, uint64_t* mask, int words) {
  __shared__ int s_par[kMaxAttendBlock];
  const int r = blockIdx.x;
  for (int j = threadIdx.x; j < a.blk; j += 256) s_par[j] = a.parent[(int64_t)r * a.blk + j];
  __syncthreads();
  for (int j = threadIdx.x; j < a.blk; j += 256) {
    uint64_t* out = mask + ((int64_t)r * a.blk + j) * words;
    int i = j;
    for (int w = words - 1; w >= 0; --w) {  // parents come before their children
      uint64_t bits = 0;
      while (i >= 64 * w) {
        bits |= 1ull << (i & 63);
        const int p = s_par[i];
        i = p < i ? p : -1;  // a bad parent ends the path
      }
      out[w] = bits;
    }
  }
}

// An item is four rows of one head of a job that starts in one share and ends in a later one; its parts
// are added in order, a lane the same 16 bytes of each.  WIDE (few jobs, many parts each): a block per
// item, its eight waves take every eighth part and are added at the end (4 lines of 125 000 8-bit
// positions, 64 parts a job: 2 us less than with four waves).  Otherwise a wave per item.  The items are
// counted by jobs, where there are fewer of those than shares (3 lines of 32 rows: 17 us less; most
// shares' items would be empty).  Blocks behind the items: the status of one line each.
constexpr int join_waves(bool wide) { return wide ? 8 : 4; }

// the parts first, first + stride, ... of rows row0 .. row0+3 (live of them)
template <int DP, bool WIDE> struct JoinSum {
  static constexpr int NV = kJoinRows * DP / 4 / 64;  // 16-byte pieces per lane
  f32x4 o[NV];
  float m[NV], l[NV];
  __device__ void run(const AttendKernelArgs& k, const AttendInfo& in, int w, int hi, int row0, int live,
                      int first, int stride) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      o[v] = f32x4{0, 0, 0, 0};
      m[v] = kNegBig;
      l[v] = 0.0f;
    }
    constexpr int kAhead = (WIDE ? 8 : 4) / (DP > 128 ? 2 : 1);  // parts loaded together
    for (int p0 = first; p0 < in.parts; p0 += stride * kAhead) {
      f32x4 y[kAhead][NV];
      float2 ml[kAhead][NV];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {  // no branches: past the last part, the last again
        const int p = min(p0 + stride * u, in.parts - 1);
        const int64_t slot = p == 0 ? in.slot : 2 * (int64_t)(w + p);
        const int64_t at = (slot * k.hpj + hi) * k.prow + row0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int e = (v * 64 + lane) * 4, row = e / DP, ok = min(row, live - 1);
          ml[u][v] = k.ml[at + ok];
          y[u][v] = *reinterpret_cast<const f32x4*>(k.o + (at + ok) * DP + (e - row * DP));
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const bool on = p0 + stride * u < in.parts;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const float mx = fmaxf(m[v], ml[u][v].x);
          const float f0 = __builtin_amdgcn_exp2f(m[v] - mx);
          const float f1 = __builtin_amdgcn_exp2f(ml[u][v].x - mx);
          // selected, not multiplied by zero: a part may hold infinities
          o[v] = on ? o[v] * f0 + y[u][v] * f1 : o[v];
          l[v] = on ? l[v] * f0 + ml[u][v].y * f1 : l[v];
          m[v] = on ? mx : m[v];
        }
      }
    }
  }
};

template <typename T, int DP, bool WIDE>
__global__ __launch_bounds__(64 * join_waves(WIDE)) void k_attend_join(AttendKernelArgs k, int rows,
                                                                   int items, int f8) {
  constexpr int kJoinWaves = join_waves(WIDE);
  typedef JoinSum<DP, WIDE> Sum;
  __shared__ f32x4 s_o[WIDE ? kJoinWaves : 1][kJoinRows * DP / 4];
  __shared__ float s_m[kJoinWaves][kJoinRows], s_l[kJoinWaves][kJoinRows];
  const AttendArgs& a = k.a;
  const psispec_paged_cache& c = a.c;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int quads = k.prow / kJoinRows;
  const int item_blocks = WIDE ? items : (items + kJoinWaves - 1) / kJoinWaves;
  if ((int)blockIdx.x >= item_blocks) {
    const int r = blockIdx.x - item_blocks;
    int L, n;
    bool bad = !line_rows(a.len, a.n_new, r, a.blk, c.slots, c.page_size, &L, &n), badp = false;
    if (!bad && n > 0) {
      const int32_t* tab = c.table + (int64_t)r * c.table_stride;
      const int last = (int)(((int64_t)L + n - 1) / c.page_size);
      for (int s = threadIdx.x; s <= last; s += 64 * kJoinWaves)
        bad |= (uint32_t)tab[s] >= (uint32_t)c.num_pages;
      if (a.parent)
        for (int j = threadIdx.x; j < n; j += 64 * kJoinWaves) {
          const int p = a.parent[(int64_t)r * a.blk + j];
          badp |= p < -1 || p >= j;
        }
    }
    const bool b0 = __syncthreads_or(bad), b1 = __syncthreads_or(badp);
    if (threadIdx.x == 0)
      a.status[r] = (b0 ? PSISPEC_ST_BAD_PAGE : 0) | (b1 ? PSISPEC_ST_BAD_PARENT : 0);
    return;
  }
  const int item = WIDE ? blockIdx.x : blockIdx.x * kJoinWaves + wave;
  if (item >= items) return;
  const int at = item / (k.hpj * quads);
  const int hi = (item - at * k.hpj * quads) / quads;
  const int row0 = (item % quads) * kJoinRows;
  int L, n;
  if (k.by_job && (!line_rows(a.len, a.n_new, at / (k.hgroups * k.nmt), a.blk, c.slots, c.page_size, &L,
                              &n) ||
                   at % k.nmt * rows >= n * k.G))
    return;  // no step, no info
  const AttendInfo in = k.info[at];
  if (in.parts == 0) return;
  line_rows(a.len, a.n_new, in.r, a.blk, c.slots, c.page_size, &L, &n);
  const int live = min(n * k.G - in.mt * rows, rows) - row0;  // live rows from row0 on
  if (live <= 0) return;
  const int h = in.h * k.hpj + hi;
  const float vs = f8 && c.v_scale ? c.v_scale[h] : 1.0f;
  auto store = [&](int e, f32x4 y, float l) {  // 16 bytes e of the four rows
    const int row = e * 4 / DP, d = e * 4 - row * DP;
    if (row >= live || d >= c.dim) return;
    const int q = in.mt * rows + row0 + row, i = q / k.G;
    const float f = vs / l;
    typename attend::Elem<T>::x4 z;
#pragma unroll
    for (int u = 0; u < 4; ++u) z[u] = (T)(y[u] * f);
    T* out = static_cast<T*>(a.out) + ((int64_t)in.r * a.blk + i) * a.out_stride +
             (int64_t)(h * k.G + (q - i * k.G)) * c.dim + d;
    *reinterpret_cast<typename attend::Elem<T>::x4*>(out) = z;
  };
  Sum sum;
  sum.run(k, in, in.w, hi, row0, live, WIDE ? wave : 0, WIDE ? kJoinWaves : 1);
  if constexpr (!WIDE) {
#pragma unroll
    for (int v = 0; v < Sum::NV; ++v) store(v * 64 + lane, sum.o[v], sum.l[v]);
  } else {
#pragma unroll
    for (int v = 0; v < Sum::NV; ++v) {
      const int e = v * 64 + lane;
      s_o[wave][e] = sum.o[v];
      if (e * 4 % DP == 0) {
        s_m[wave][e * 4 / DP] = sum.m[v];
        s_l[wave][e * 4 / DP] = sum.l[v];
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kJoinRows * DP / 4; e += 64 * kJoinWaves) {
      const int row = e * 4 / DP;
      float mx = kNegBig, l = 0.0f;
      for (int u = 0; u < kJoinWaves; ++u) mx = fmaxf(mx, s_m[u][row]);
      f32x4 y = {0, 0, 0, 0};
      for (int u = 0; u < kJoinWaves; ++u) {
        const float f = __builtin_amdgcn_exp2f(s_m[u][row] - mx);
        y += s_o[u][e] * f;
        l += s_l[u][row] * f;
      }
      store(e, y, l);
    }
  }
}

template <typename T, int DP>
hipError_t launch_join_dp(const AttendKernelArgs& k, const AttendPlan& p, bool whole,
                          hipStream_t stream) {
  const int64_t jobs = (int64_t)k.a.batch * k.hgroups * k.nmt;
  const int rows = p.mt * 16, items = whole ? 0 : (k.by_job ? (int)jobs : k.used) * k.hpj * (p.prow / kJoinRows);
  const int f8 = k.a.c.dtype == PSISPEC_F8E4M3;
  const int status = k.a.status ? k.a.batch : 0;
  // Many parts per job, and no more items than CUs: 16 lines of one row (128 items of 16 parts) 5.4 us wide,
  // 7.3 otherwise; 8 lines of 9 rows (576 items of 8 parts) 9.8 and 4.8, 4 lines (288 of 16) 7.7 and 4.9.
  if (jobs * 8 <= k.shares && items <= kAttendCUs)
    PSISPEC_LAUNCH("attend_join", (k_attend_join<T, DP, true>), dim3((unsigned)(items + status)),
                   dim3(64 * join_waves(true)), 0, stream, k, rows, items, f8);
  else
    PSISPEC_LAUNCH("attend_join", (k_attend_join<T, DP, false>),
                   dim3((unsigned)((items + join_waves(false) - 1) / join_waves(false) + status)),
                   dim3(64 * join_waves(false)), 0, stream, k, rows, items, f8);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_join(const AttendKernelArgs& k, const AttendPlan& p, bool whole, hipStream_t stream) {
  return p.dp == 64    ? launch_join_dp<T, 64>(k, p, whole, stream)
         : p.dp == 128 ? launch_join_dp<T, 128>(k, p, whole, stream)
                       : launch_join_dp<T, 256>(k, p, whole, stream);
}

}  // namespace

size_t attend_workspace_bytes(int batch, int blk, int heads_q, int heads_kv, int dim) {
  return make_attend_plan(batch, blk, heads_q, heads_kv, dim).total;
}

hipError_t launch_attend(const AttendArgs& a, psispec_dtype dtype, void* workspace,
                         hipStream_t stream) {
  const AttendPlan p = make_attend_plan(a.batch, a.blk, a.heads_q, a.c.heads, a.c.dim);
  const bool f8 = a.c.dtype == PSISPEC_F8E4M3;
  char* ws = static_cast<char*>(workspace);
  AttendKernelArgs k{};
  k.a = a;
  k.G = a.heads_q / a.c.heads;
  k.nmt = p.nmt;
  k.mask_words = p.mask_words;
  // Short lines: a job is one step, so no border cuts it.
  const int64_t most = (int64_t)a.c.slots * a.c.page_size;
  const bool few = p.hpj > 1 && p.sub == 1 && (int64_t)a.batch * a.c.heads <= kFewHeads;
  const bool whole = most <= (few ? kWholeFewPositions : kWholePositions);
  int mt = p.mt;
  if (whole) {
    const int64_t rows = (int64_t)a.blk * k.G;
    const int solo_mt = rows > 16 && p.dp <= 128 ? 2 : 1;
    const int64_t solo_nmt = (rows + 16 * solo_mt - 1) / (16 * solo_mt);
    const int64_t jobs = a.batch * a.c.heads * solo_nmt;
    k.solo = jobs >= 2 * p.wgs && (most <= kSoloPositions || solo_nmt == p.nmt);
    if (k.solo) {
      mt = solo_mt;
      k.nmt = (int)solo_nmt;
    }
  }
  k.hpj = whole ? 1 : p.hpj;
  k.hgroups = a.c.heads / k.hpj;
  k.shares = whole ? p.wgs : p.wgs / p.sub;
  k.skew = p.wgs > kAttendCUs && !whole ? 2 : 0;  // whole jobs do not divide so: 119 -> 110 us for that case
  k.prow = p.prow;
  const int step = kAttendTile * (k.solo ? 1 : kAttendWaves);
  k.step_tiles = whole ? (int)((most + step - 1) / step) : 1;
  // a job's own cost in steps (queries and page ids fetched, the waves joined): 64 lines of 9 rows 120.0 us
  // with 3, 120.5 with 2, 121.1 with 4, 124.4 with 6; a wave that has the head to itself joins nothing
  k.job_cost = whole ? 0 : p.hpj > 1 && p.sub == 1 ? 1 : 3;
  // no more workgroups than there can be units
  const int tiles = (p.sub > 1 ? kAttendWaves : kAttendWaves / k.hpj) * k.step_tiles;
  const int64_t steps = (most + tiles * kAttendTile - 1) / (tiles * kAttendTile);
  const int64_t units = (steps + k.job_cost) * k.hgroups * k.nmt * a.batch;
  k.used = (int)(units < k.shares ? units : k.shares);
  k.by_job = !whole && (int64_t)a.batch * k.hgroups * k.nmt <= k.shares;
  k.ps_magic = (uint32_t)(((uint64_t(1) << 32) + a.c.page_size - 1) / a.c.page_size);
  const int es = f8 ? 1 : 2;
  const int64_t page_bytes = a.c.page_stride * es, row_bytes = a.c.row_stride * es;
  k.halves = a.c.dim == p.dp && a.c.page_size % 16 == 0 && page_bytes < (int64_t(1) << 31) &&
             row_bytes * (a.c.page_size + 16) < (int64_t(1) << 31);
  if (k.halves) {
    k.page_bytes = (uint32_t)page_bytes;
    k.row_bytes = (uint32_t)row_bytes;
  }
  k.c = a.scale * kLog2e;
  k.info = reinterpret_cast<AttendInfo*>(ws);
  k.ml = reinterpret_cast<float2*>(ws + p.off_ml);
  k.o = reinterpret_cast<float*>(ws + p.off_o);
  if (a.parent) {
    uint64_t* mask = reinterpret_cast<uint64_t*>(ws + p.off_mask);
    k.mask = mask;
    PSISPEC_LAUNCH("tree_mask", k_tree_mask, dim3((unsigned)a.batch), dim3(256), 0, stream, a, mask,
                   p.mask_words);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipError_t e;
  if (dtype == PSISPEC_BF16)
    e = f8 ? launch_attend_bf16_f8(k, p.dp, mt, stream) : launch_attend_bf16(k, p.dp, mt, stream);
  else
    e = f8 ? launch_attend_f16_f8(k, p.dp, mt, stream) : launch_attend_f16(k, p.dp, mt, stream);
  if (e != hipSuccess) return e;
  if (whole && !a.status) return hipSuccess;
  return dtype == PSISPEC_BF16 ? launch_join<__bf16>(k, p, whole, stream)
                               : launch_join<_Float16>(k, p, whole, stream);
}

}  // namespace psispec
