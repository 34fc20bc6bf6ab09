// pages.hip -- pages of a KV cache: the commit of a verified block, forks, cuts and frees of lines by
// shared pages, and pages for the next block (with the copy on a first write after a fork).
//
// State: table[r][s] names the page of positions [s ps, (s+1) ps) of line r (-1: none); refs[p] is the
// number of table entries that name page p; a page is free exactly when refs[p] = 0.  There is no
// list of free pages to keep in step: the reserve takes the lowest-numbered pages with count 0, so
// the outcome depends on tables and counts alone and not on the order of earlier calls.
#include "paged.h"

namespace psispec {
namespace {

constexpr int kPgThreads = 256;
constexpr int kScanChunk = 4096;      // pages whose counts one workgroup scans
constexpr int kMaxChunks = 4096;      // 16.8 M pages

__device__ inline bool page_ok(int p, int num_pages) { return (uint32_t)p < (uint32_t)num_pages; }

// ------------------------------------------------------------------------------------------------
// commit: kept row i of line r moves from position len + keep[i] to len + i, keep strictly
// increasing.  As in the contiguous commit the move is in place and safe in increasing i: a thread
// owns a few 16-byte slices of every row, and the source of every later row lies behind row i.  Rows
// already in place are dropped from the list that the block builds in LDS.  Bound by HBM for large
// batches, by the chain count -> list -> pages -> rows for small ones.
// ------------------------------------------------------------------------------------------------
constexpr int kCommitBatch = 8;       // rows loaded before they are stored
constexpr int kCommitSlices = 2;      // 16-byte slices of a row per thread (1 slice: 87 us for 256 lines,
                                      // 2: 44, 4: 45, 8: 51)

struct Move {
  int64_t src, dst;  // byte offsets within a plane
};

// The line's commit is valid (PSISPEC_ST_* otherwise): counts, order and pages.  Every thread of the
// block returns the same; the rows that move are in s_mv[0 .. *moves-1], in order.
__device__ inline int commit_check(const PagedCommitArgs& a, int r, int* s_keep, Move* s_mv,
                                   int* s_cnt, int* moves) {
  const int n = a.n_keep[r], L = a.len[r];
  const int nk = a.keep ? min(a.keep_stride, a.blk) : 0;
  for (int i = threadIdx.x; i < nk; i += blockDim.x)
    s_keep[i] = a.keep[(int64_t)r * a.keep_stride + i];
  if (threadIdx.x == 0) *s_cnt = 0;
  __syncthreads();
  const int ps = a.pool.page_size;
  const int64_t most = (int64_t)a.slots * ps;  // a short block may end at the table's end: blk need not fit
  bool bad = n < 0 || n > a.blk || L < 0 || (int64_t)L + n > most || (a.keep && n > a.keep_stride);
  bool badpage = false;
  if (!bad && a.keep) {
    const int32_t* tab = a.table + (int64_t)r * a.table_stride;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int k = s_keep[i], kp = i == 0 ? -1 : s_keep[i - 1];
      if (k < 0 || k >= a.blk || k <= kp || (int64_t)L + k >= most) {
        bad = true;
      } else if (k != i) {
        // keep is strictly increasing from keep[0] >= 0, so once keep[i] > i every later row moves
        const int ss = (L + k) / ps, ds = (L + i) / ps;
        const int sp = tab[ss], dp = tab[ds];
        badpage |= !page_ok(sp, a.pool.num_pages) || !page_ok(dp, a.pool.num_pages);
        s_mv[i].src = sp * a.pool.page_stride + (int64_t)(L + k - ss * ps) * a.pool.row_bytes;
        s_mv[i].dst = dp * a.pool.page_stride + (int64_t)(L + i - ds * ps) * a.pool.row_bytes;
        atomicAdd(s_cnt, 1);
      }
    }
  }
  const bool any_bad = __syncthreads_or(bad);
  const bool any_page = __syncthreads_or(badpage);
  *moves = *s_cnt;
  return any_bad ? PSISPEC_ST_BAD_KEEP : any_page ? PSISPEC_ST_BAD_PAGE : 0;
}

// with_len: tile 0 writes the line's status and new length, which must not be `len` itself then.
__global__ __launch_bounds__(kPgThreads) void k_paged_commit(PagedCommitArgs a, int ntiles,
                                                             int with_len) {
  extern __shared__ char smem[];
  __shared__ int s_cnt;
  Move* s_mv = reinterpret_cast<Move*>(smem);
  int* s_keep = reinterpret_cast<int*>(s_mv + a.blk);
  const int r = blockIdx.x / ntiles;
  const int tile = blockIdx.x - r * ntiles;
  int moves;
  const int st = commit_check(a, r, s_keep, s_mv, &s_cnt, &moves);
  const int n = a.n_keep[r];
  if (with_len && tile == 0 && threadIdx.x == 0) {
    const int L = a.len[r];
    a.new_len[r] = st ? L : L + n;
    if (a.status) a.status[r] = st;
  }
  if (st || moves == 0) return;
  const int64_t per_plane = a.pool.row_bytes / 16, all = per_plane * a.pool.planes;
  int64_t s = (int64_t)tile * kPgThreads * kCommitSlices + threadIdx.x;
  char* base[kCommitSlices];
  bool on[kCommitSlices];
#pragma unroll
  for (int k = 0; k < kCommitSlices; ++k, s += kPgThreads) {
    on[k] = s < all;
    const int64_t w = (on[k] ? s : 0) / per_plane;
    base[k] = static_cast<char*>(a.pool.base) + w * a.pool.plane_stride +
              ((on[k] ? s : 0) - w * per_plane) * 16;
  }
  for (int i0 = n - moves; i0 < n; i0 += kCommitBatch) {  // the moving rows are the last ones
    u32x4 v[kCommitBatch][kCommitSlices] = {};
#pragma unroll
    for (int u = 0; u < kCommitBatch; ++u) {
      if (i0 + u < n) {
        const int64_t src = s_mv[i0 + u].src;
#pragma unroll
        for (int k = 0; k < kCommitSlices; ++k)
          if (on[k]) v[u][k] = *reinterpret_cast<const u32x4*>(base[k] + src);
      }
    }
#pragma unroll
    for (int u = 0; u < kCommitBatch; ++u) {
      if (i0 + u < n) {
        const int64_t dst = s_mv[i0 + u].dst;
#pragma unroll
        for (int k = 0; k < kCommitSlices; ++k)
          if (on[k]) *reinterpret_cast<u32x4*>(base[k] + dst) = v[u][k];
      }
    }
  }
}

// New lengths and status alone: no row moves, or the new lengths overwrite the old ones, which every
// block of the move reads.
__global__ __launch_bounds__(64) void k_paged_len(PagedCommitArgs a) {
  extern __shared__ char smem[];
  __shared__ int s_cnt;
  Move* s_mv = reinterpret_cast<Move*>(smem);
  int* s_keep = reinterpret_cast<int*>(s_mv + a.blk);
  const int r = blockIdx.x;
  int moves;
  const int st = commit_check(a, r, s_keep, s_mv, &s_cnt, &moves);
  if (threadIdx.x == 0) {
    const int L = a.len[r];
    a.new_len[r] = st ? L : L + a.n_keep[r];
    if (a.status) a.status[r] = st;
  }
}

// ------------------------------------------------------------------------------------------------
// assign: line r becomes the first new_len[r] positions of the old line src[r].
// ------------------------------------------------------------------------------------------------

// What line r becomes, but for the pages taken, which are looked at with the entries.
struct AssignLine {
  int from, cut, want;  // the line that entries 0 .. cut-1 come from, the new length
  bool bad;
};
__device__ inline AssignLine assign_begin(const AssignArgs& a, int r) {
  AssignLine l;
  const int src = a.src[r];
  l.want = src == -1 ? 0 : a.new_len[r];
  l.bad = src < -1 || src >= a.batch || l.want < 0;
  l.cut = 0;
  if (!l.bad && src >= 0) {
    l.bad = l.want > a.len[src] || (int64_t)l.want > (int64_t)a.slots * a.page_size;
    l.cut = l.bad ? 0 : (int)(((int64_t)l.want + a.page_size - 1) / a.page_size);
  }
  l.from = l.bad || src < 0 ? r : src;
  return l;
}

// One workgroup per line: the new entries into the workspace and the changes of the counts (integer
// adds: the sums do not depend on their order); then k_assign_write, for a line's old entries are read
// by others.
__global__ __launch_bounds__(kPgThreads) void k_assign_count(AssignArgs a, int32_t* newtab,
                                                             int32_t* newlen) {
  const int r = blockIdx.x;
  const AssignLine l = assign_begin(a, r);
  const int32_t* from = a.table + (int64_t)l.from * a.table_stride;
  const int32_t* old = a.table + (int64_t)r * a.table_stride;
  bool bad = l.bad;
  for (int s = threadIdx.x; s < l.cut; s += kPgThreads) bad |= !page_ok(from[s], a.num_pages);
  bad = __syncthreads_or(bad);
  for (int s = threadIdx.x; s < a.slots; s += kPgThreads) {
    const int o = old[s];
    const int e = bad ? o : s < l.cut ? from[s] : -1;
    newtab[(int64_t)r * a.slots + s] = e;
    if (e != o) {
      if (page_ok(e, a.num_pages)) atomicAdd(&a.refs[e], 1);
      if (page_ok(o, a.num_pages)) atomicSub(&a.refs[o], 1);
    }
  }
  if (threadIdx.x == 0) {
    newlen[r] = bad ? a.len[r] : l.want;
    if (a.status) a.status[r] = bad ? PSISPEC_ST_BAD_PAGE : 0;
  }
}

__global__ __launch_bounds__(kPgThreads) void k_assign_write(AssignArgs a, const int32_t* newtab,
                                                             const int32_t* newlen) {
  const int r = blockIdx.x;
  for (int s = threadIdx.x; s < a.slots; s += kPgThreads)
    a.table[(int64_t)r * a.table_stride + s] = newtab[(int64_t)r * a.slots + s];
  if (threadIdx.x == 0) a.len[r] = newlen[r];
}

// Few entries in one launch of one workgroup: each thread holds its old and new entries in registers,
// and a barrier lies between the reads of the old tables and the writes of the new ones.  64 lines of 39
// slots: 4.5 us against 4.7 + 4.4 in two launches; 128 of 57: 10.7 (one CU's atomics) against 4.3 + 4.3.
constexpr int kOneBlock = 1024;
constexpr int kOneEntries = 4;  // per thread
__global__ __launch_bounds__(kOneBlock) void k_assign_one(AssignArgs a) {
  __shared__ int s_from[kOneBlock], s_cut[kOneBlock], s_bad[kOneBlock];
  const int tid = threadIdx.x;
  int len_new = 0;
  if (tid < a.batch) {
    const AssignLine l = assign_begin(a, tid);
    s_from[tid] = l.from;
    s_cut[tid] = l.cut;
    s_bad[tid] = l.bad;
    len_new = l.want;
  }
  __syncthreads();
  const int all = a.batch * a.slots;
  int line[kOneEntries], old[kOneEntries], now[kOneEntries];
#pragma unroll
  for (int k = 0; k < kOneEntries; ++k) {
    const int x = tid + k * kOneBlock;
    line[k] = -1;
    if (x < all) {
      const int r = x / a.slots, t = x - r * a.slots;
      line[k] = r;
      old[k] = a.table[(int64_t)r * a.table_stride + t];
      now[k] = t < s_cut[r] ? a.table[(int64_t)s_from[r] * a.table_stride + t] : -1;
      if (t < s_cut[r] && !page_ok(now[k], a.num_pages)) s_bad[r] = 1;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kOneEntries; ++k) {
    if (line[k] < 0 || s_bad[line[k]] || old[k] == now[k]) continue;
    const int t = tid + k * kOneBlock - line[k] * a.slots;
    if (page_ok(now[k], a.num_pages)) atomicAdd(&a.refs[now[k]], 1);
    if (page_ok(old[k], a.num_pages)) atomicSub(&a.refs[old[k]], 1);
    a.table[(int64_t)line[k] * a.table_stride + t] = now[k];
  }
  if (tid < a.batch) {
    if (!s_bad[tid]) a.len[tid] = len_new;
    if (a.status) a.status[tid] = s_bad[tid] ? PSISPEC_ST_BAD_PAGE : 0;
  }
}

// ------------------------------------------------------------------------------------------------
// reserve
// ------------------------------------------------------------------------------------------------

// Exclusive sum over the block's 256 threads; *total = the block's sum.  s: 4 ints of LDS.
__device__ inline int block_excl_sum(int x, int* s, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(inc, o, 64);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 63) s[wave] = inc;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPgThreads / 64; ++w) {
    before += w < wave ? s[w] : 0;
    all += s[w];
  }
  *total = all;
  return before + inc - x;
}

struct ReserveWs {
  int32_t* need;   // [batch] pages that the line needs; -1: invalid
  int32_t* first;  // [batch] pages that the lines before it need; -1: the free ones do not reach it
  int32_t* take;   // [batch][J] per slot: kNoNeed, -1 (no page there) or the shared page to replace
  int32_t* cnt;    // [chunks] free pages per chunk
  int32_t* ids;    // [batch * J] the free pages to hand out, in order
  int J, chunks;
};
constexpr int kNoNeed = -2;

// Sum over x[0 .. n-1] (negative entries count as 0) by the whole block.
__device__ inline int block_sum_of(const int32_t* x, int n, int* s) {
  int part = 0, total;
  for (int k = threadIdx.x; k < n; k += kPgThreads) part += max(x[k], 0);
  block_excl_sum(part, s, &total);
  return total;
}

// What line r needs in slot j from its first touched slot on (m of them): w.take[r][j], 1 if a page.
__device__ inline int reserve_slot(const ReserveArgs& a, const ReserveWs& w, int r, int j, int s0, int m,
                                   int L, bool* bad) {
  const int np = a.pool.num_pages;
  int t = kNoNeed;
  if (j < m) {
    const int p = a.table[(int64_t)r * a.table_stride + s0 + j];
    // a slot that already holds rows of the line must have its page
    *bad |= p >= np || (p < 0 && j == 0 && L > s0 * a.pool.page_size);
    t = p < 0 ? -1 : page_ok(p, np) && a.refs[p] > 1 ? p : kNoNeed;
  }
  w.take[(int64_t)r * w.J + j] = t;
  return t != kNoNeed;
}
__device__ inline bool reserve_span(const ReserveArgs& a, int r, int* L, int* s0, int* m) {
  int rows;
  const bool ok = line_rows(a.len, a.n_new, r, a.blk, a.slots, a.pool.page_size, L, &rows);
  *s0 = ok ? *L / a.pool.page_size : 0;
  *m = ok && rows > 0 ? (*L + rows - 1) / a.pool.page_size - *s0 + 1 : 0;
  return ok;
}

// Block r < batch: what line r needs.  Block batch + c: the number of free pages in chunk c.
__global__ __launch_bounds__(kPgThreads) void k_reserve_plan(ReserveArgs a, ReserveWs w) {
  __shared__ int s_sum[4];
  int n = 0, total;
  if ((int)blockIdx.x >= a.batch) {
    const int c = blockIdx.x - a.batch;
    for (int k = threadIdx.x; k < kScanChunk; k += kPgThreads) {
      const int p = c * kScanChunk + k;
      n += p < a.pool.num_pages && a.refs[p] == 0;
    }
    block_excl_sum(n, s_sum, &total);
    if (threadIdx.x == 0) w.cnt[c] = total;
    return;
  }
  const int r = blockIdx.x;
  int L, s0, m;
  bool bad = !reserve_span(a, r, &L, &s0, &m);
  for (int j = threadIdx.x; j < w.J; j += kPgThreads) n += reserve_slot(a, w, r, j, s0, m, L, &bad);
  block_excl_sum(n, s_sum, &total);
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) w.need[r] = bad ? -1 : total;
}

// Chunk c's free pages go to their places among all free pages.
__global__ __launch_bounds__(kPgThreads) void k_reserve_ids(ReserveArgs a, ReserveWs w) {
  __shared__ int s_sum[4];
  const int c = blockIdx.x;
  const int want = block_sum_of(w.need, a.batch, s_sum);
  if (c == 0) {
    const int avail = block_sum_of(w.cnt, w.chunks, s_sum);
    int base = 0, total;
    for (int r0 = 0; r0 < a.batch; r0 += kPgThreads) {
      const int r = r0 + threadIdx.x;
      const int need = r < a.batch ? max(w.need[r], 0) : 0;
      const int first = base + block_excl_sum(need, s_sum, &total);
      if (r < a.batch) w.first[r] = need == 0 || first + need <= avail ? first : -1;
      base += total;
    }
  }
  const int before = block_sum_of(w.cnt, c, s_sum);
  if (before >= want) return;
  int n;
  constexpr int kPer = kScanChunk / kPgThreads;
  const int p0 = c * kScanChunk + threadIdx.x * kPer;
  bool fr[kPer];
  int mine = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    fr[k] = p0 + k < a.pool.num_pages && a.refs[p0 + k] == 0;
    mine += fr[k];
  }
  int at = before + block_excl_sum(mine, s_sum, &n);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (fr[k]) {
      if (at < want) w.ids[at] = p0 + k;
      ++at;
    }
  }
}

// Both in one launch of one workgroup for small pools and few slots: a line belongs to `group` lanes
// (a power of two), a wave counts the free pages of its run of the pool by votes.  128 lines, 7300 pages:
// 6.3 us against 4.4 + 6.0.
constexpr int kOneChunks = 8;
constexpr int kOneSlots = 4;  // slots per lane
__global__ __launch_bounds__(kOneBlock) void k_reserve_one(ReserveArgs a, ReserveWs w, int log_group) {
  constexpr int kWaves = kOneBlock / 64, kVotes = kOneChunks * kScanChunk / kOneBlock;
  __shared__ int s_free[kWaves], s_need[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int group = 1 << log_group, r = tid >> log_group;
  int n = 0, bad = 0;
  if (r < a.batch) {
    int L, s0, m;
    bool b = !reserve_span(a, r, &L, &s0, &m);
    for (int j = tid & (group - 1); j < w.J; j += group) n += reserve_slot(a, w, r, j, s0, m, L, &b);
    bad = b;
  }
  const int votes = w.chunks * (kScanChunk / kOneBlock);
  const int p0 = wave * votes * 64 + lane;
  uint64_t fr[kVotes];
  int mine = 0;
#pragma unroll
  for (int k = 0; k < kVotes; ++k) {
    fr[k] = 0;
    if (k < votes) {
      const int p = p0 + 64 * k;
      fr[k] = __ballot(p < a.pool.num_pages && a.refs[min(p, a.pool.num_pages - 1)] == 0);
      mine += __popcll(fr[k]);
    }
  }
  for (int o = 1; o < group; o <<= 1) {
    n += __shfl_xor(n, o, 64);
    bad |= __shfl_xor(bad, o, 64);
  }
  const bool first_lane = (tid & (group - 1)) == 0 && r < a.batch;
  const int need = first_lane && !bad ? n : 0;
  int upto = need;  // what the lines up to this one need
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(upto, o, 64);
    if (lane >= o) upto += y;
  }
  if (lane == 0) s_free[wave] = mine;
  if (lane == 63) s_need[wave] = upto;
  __syncthreads();
  int at = 0, avail = 0, want = 0;
  for (int v = 0; v < kWaves; ++v) {
    at += v < wave ? s_free[v] : 0;
    upto += v < wave ? s_need[v] : 0;
    avail += s_free[v];
    want += s_need[v];
  }
  if (first_lane) {
    w.need[r] = bad ? -1 : need;
    w.first[r] = need == 0 || upto <= avail ? upto - need : -1;
  }
#pragma unroll
  for (int k = 0; k < kVotes; ++k) {
    if (k >= votes || at >= want) break;
    const int to = at + __popcll(fr[k] & ((1ull << lane) - 1));
    if ((fr[k] >> lane & 1) && to < want) w.ids[to] = p0 + 64 * k;
    at += __popcll(fr[k]);
  }
}

// Workgroup (r, tile): tile 0 writes the line's entries, counts and status; every tile copies its
// part of the shared tail page.
constexpr int kCopyLoads = 4;
constexpr int kCopyTile = kPgThreads * 16 * kCopyLoads;

__global__ __launch_bounds__(kPgThreads) void k_reserve_apply(ReserveArgs a, ReserveWs w,
                                                              int tiles_per_plane) {
  __shared__ int s_sum[4];
  const int tiles = tiles_per_plane * a.pool.planes;
  const int r = blockIdx.x / tiles;
  const int tile = blockIdx.x - r * tiles;
  const int need = w.need[r], first = w.first[r];
  const bool served = first >= 0;
  if (tile == 0 && threadIdx.x == 0 && a.status)
    a.status[r] = need < 0 ? PSISPEC_ST_BAD_PAGE : served ? 0 : PSISPEC_ST_NO_PAGE;
  if (need <= 0 || !served) return;
  const int L = a.len[r], ps = a.pool.page_size;
  const int s0 = L / ps, rem = L - s0 * ps;
  const int32_t* take = w.take + (int64_t)r * w.J;
  if (tile == 0) {
    int base = first, total;
    for (int j0 = 0; j0 < w.J; j0 += kPgThreads) {
      const int j = j0 + threadIdx.x;
      const int t = j < w.J ? take[j] : kNoNeed;
      const int k = base + block_excl_sum(t != kNoNeed, s_sum, &total);
      if (t != kNoNeed) {
        const int p = w.ids[k];
        a.table[(int64_t)r * a.table_stride + s0 + j] = p;
        atomicAdd(&a.refs[p], 1);
        if (t >= 0) atomicSub(&a.refs[t], 1);
      }
      base += total;
    }
  }
  const int old = take[0];
  if (old < 0 || rem == 0) return;  // the tail page is the line's own, or holds none of its rows
  const int64_t bytes = rem * a.pool.row_bytes;
  const int plane = tile / tiles_per_plane;
  const int64_t at = (int64_t)(tile - plane * tiles_per_plane) * kCopyTile + threadIdx.x * 16;
  char* base = static_cast<char*>(a.pool.base) + plane * a.pool.plane_stride + at;
  const char* src = base + old * a.pool.page_stride;
  char* dst = base + w.ids[first] * a.pool.page_stride;
  u32x4 v[kCopyLoads] = {};
#pragma unroll
  for (int k = 0; k < kCopyLoads; ++k)
    if (at + k * kPgThreads * 16 < bytes)
      v[k] = *reinterpret_cast<const u32x4*>(src + k * kPgThreads * 16);
#pragma unroll
  for (int k = 0; k < kCopyLoads; ++k)
    if (at + k * kPgThreads * 16 < bytes)
      *reinterpret_cast<u32x4*>(dst + k * kPgThreads * 16) = v[k];
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// slots of a line that n <= blk rows can touch
int reserve_slots(int blk, int page_size, int slots) {
  const int j = (blk - 1) / page_size + 2;
  return j < slots ? j : slots;
}

}  // namespace

size_t pages_workspace_bytes(int batch, int slots, int num_pages, int blk, int page_size) {
  const size_t assign = up256(sizeof(int32_t) * (size_t)batch * slots) + up256(sizeof(int32_t) * batch);
  const size_t J = reserve_slots(blk, page_size, slots);
  const size_t chunks = ((size_t)num_pages + kScanChunk - 1) / kScanChunk;
  if (chunks > kMaxChunks || batch * J > (size_t)1 << 30) return 0;
  const size_t reserve = 2 * up256(sizeof(int32_t) * batch) +
                         2 * up256(sizeof(int32_t) * batch * J) + up256(sizeof(int32_t) * chunks);
  return (assign > reserve ? assign : reserve) + 256;
}

hipError_t launch_paged_commit(const PagedCommitArgs& a, hipStream_t stream) {
  const int64_t slices = a.pool.planes * (a.pool.row_bytes / 16);
  const int per = kPgThreads * kCommitSlices;
  const int ntiles = (int)((slices + per - 1) / per);
  const size_t shm = a.blk * (sizeof(Move) + sizeof(int));
  // the two arrays of lengths apart: one launch
  const int apart = a.new_len != a.len;
  if (a.keep) {  // without a list the kept rows are in place
    PSISPEC_LAUNCH("paged_commit", k_paged_commit, dim3((unsigned)((int64_t)a.batch * ntiles)),
                   dim3(kPgThreads), shm, stream, a, ntiles, apart);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || apart) return e;
  }
  PSISPEC_LAUNCH("paged_len", k_paged_len, dim3((unsigned)a.batch), dim3(64), shm, stream, a);
  return hipGetLastError();
}

hipError_t launch_pages_assign(const AssignArgs& a, void* workspace, hipStream_t stream) {
  int32_t* newtab = static_cast<int32_t*>(workspace);
  int32_t* newlen = reinterpret_cast<int32_t*>(
      static_cast<char*>(workspace) + up256(sizeof(int32_t) * (size_t)a.batch * a.slots));
  if (a.batch <= kOneBlock && (int64_t)a.batch * a.slots <= kOneBlock * kOneEntries) {
    PSISPEC_LAUNCH("assign_one", k_assign_one, dim3(1), dim3(kOneBlock), 0, stream, a);
    return hipGetLastError();
  }
  PSISPEC_LAUNCH("assign_count", k_assign_count, dim3((unsigned)a.batch), dim3(kPgThreads), 0, stream,
                 a, newtab, newlen);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  PSISPEC_LAUNCH("assign_write", k_assign_write, dim3((unsigned)a.batch), dim3(kPgThreads), 0, stream,
                 a, newtab, newlen);
  return hipGetLastError();
}

hipError_t launch_pages_reserve(const ReserveArgs& a, void* workspace, hipStream_t stream) {
  ReserveWs w{};
  w.J = reserve_slots(a.blk, a.pool.page_size, a.slots);
  w.chunks = (a.pool.num_pages + kScanChunk - 1) / kScanChunk;
  char* at = static_cast<char*>(workspace);
  auto carve = [&](size_t n) {
    int32_t* p = reinterpret_cast<int32_t*>(at);
    at += up256(sizeof(int32_t) * n);
    return p;
  };
  w.need = carve(a.batch);
  w.first = carve(a.batch);
  w.take = carve((size_t)a.batch * w.J);
  w.ids = carve((size_t)a.batch * w.J);
  w.cnt = carve(w.chunks);
  hipError_t e;
  int lg = 6;
  while (lg > 0 && (int64_t)a.batch << lg > kOneBlock) --lg;
  if (w.chunks <= kOneChunks && a.batch <= kOneBlock && w.J <= kOneSlots << lg) {
    PSISPEC_LAUNCH("reserve_one", k_reserve_one, dim3(1), dim3(kOneBlock), 0, stream, a, w, lg);
  } else {
    PSISPEC_LAUNCH("reserve_plan", k_reserve_plan, dim3((unsigned)(a.batch + w.chunks)),
                   dim3(kPgThreads), 0, stream, a, w);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    PSISPEC_LAUNCH("reserve_ids", k_reserve_ids, dim3((unsigned)w.chunks), dim3(kPgThreads), 0, stream,
                   a, w);
  }
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int tpp = (int)((a.pool.page_size * a.pool.row_bytes + kCopyTile - 1) / kCopyTile);
  PSISPEC_LAUNCH("reserve_apply", k_reserve_apply,
                 dim3((unsigned)((int64_t)a.batch * tpp * a.pool.planes)), dim3(kPgThreads), 0, stream,
                 a, w, tpp);
  return hipGetLastError();
}

}  // namespace psispec
