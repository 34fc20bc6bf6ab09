// paged_api.hip -- the C ABI of the paged KV cache: argument checks, then the launches of append.hip,
// attend.hip and pages.hip.
#include <limits.h>
#include <math.h>

#include <initializer_list>
#include <utility>

#include "paged.h"

using namespace psispec;

namespace {

constexpr int kMaxHeads = 1024;
constexpr int64_t kMaxPositions = int64_t(1) << 30;

bool aligned(const void* p, size_t n) { return (uintptr_t)p % n == 0; }

// A grid of `blocks` workgroups can be launched: at most 2^32 - 1 threads in x, of 256 each.
bool grid_ok(int64_t blocks) { return blocks <= (int64_t(1) << 24) - 1; }

psispec_status check_cache(const psispec_paged_cache* c, psispec_dtype dtype) {
  if (!c) return PSISPEC_EINVAL;
  if (dtype != PSISPEC_BF16 && dtype != PSISPEC_F16) return PSISPEC_EDTYPE;
  if (c->dtype != (int32_t)dtype && c->dtype != PSISPEC_F8E4M3) return PSISPEC_EDTYPE;
  if (c->num_pages < 1 || c->page_size < 1 || c->page_size > kMaxPageSize || c->slots < 1 ||
      (int64_t)c->slots * c->page_size > kMaxPositions || c->table_stride < c->slots)
    return PSISPEC_EINVAL;
  if (c->heads < 1 || c->heads > kMaxHeads || c->dim < 16 || c->dim > kMaxHeadDim || c->dim % 16)
    return PSISPEC_EINVAL;
  const int64_t es = c->dtype == PSISPEC_F8E4M3 ? 1 : 2, most = int64_t(1) << 60;
  for (const int64_t s : {c->page_stride, c->row_stride, c->head_stride})
    if (s < 0 || s > most || s * es % 16) return PSISPEC_EINVAL;
  if (c->dtype != PSISPEC_F8E4M3 && (c->k_scale || c->v_scale)) return PSISPEC_EINVAL;
  return PSISPEC_OK;
}

// The places of a cache's heads in bytes: the three strides (pages, positions, heads) in increasing
// order, those of one only left out; span[i]: what the first i of them reach over, span[0] a head.
struct Places {
  int levels;
  bool apart;  // no two places share a byte: every stride is at least the span of the ones before it
  int64_t stride[3], count[3];
  __int128 span[4];
};
Places cache_places(const psispec_paged_cache* c) {
  const int64_t es = c->dtype == PSISPEC_F8E4M3 ? 1 : 2;
  int64_t stride[3] = {c->head_stride, c->row_stride, c->page_stride};
  int64_t count[3] = {c->heads, c->page_size, c->num_pages};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (stride[j] < stride[i]) {
        std::swap(stride[i], stride[j]);
        std::swap(count[i], count[j]);
      }
  Places p{};
  p.apart = true;
  p.span[0] = c->dim * es;
  for (int i = 0; i < 3; ++i) {
    if (count[i] == 1) continue;
    p.stride[p.levels] = stride[i] * es;
    p.count[p.levels] = count[i];
    p.apart &= p.stride[p.levels] >= p.span[p.levels];
    p.span[p.levels + 1] = p.span[p.levels] + (__int128)p.stride[p.levels] * (count[i] - 1);
    ++p.levels;
  }
  return p;
}

// Bytes [lo, hi) behind the first place, of the first n levels: some place has one of them.
bool bytes_in_places(const Places& p, int n, __int128 lo, __int128 hi) {
  if (hi <= 0 || lo >= p.span[n]) return false;
  if (n == 0 || !p.apart) return true;  // places within each other (read-only caches): their whole range
  const __int128 s = p.stride[n - 1], below = p.span[n - 1];
  const __int128 c0 = lo < below ? 0 : (lo - below) / s + 1;  // the first part that ends behind lo
  const __int128 c1 = (hi - 1) / s < p.count[n - 1] ? (hi - 1) / s : p.count[n - 1] - 1;
  if (c1 - c0 > 1) return true;  // a whole part in between
  for (__int128 c = c0; c <= c1; ++c)
    if (bytes_in_places(p, n - 1, lo - c * s, hi - c * s)) return true;
  return false;
}

// Places `d` bytes behind each other of the first n levels (which lie apart): some two share a byte.
bool shifted_places_meet(const Places& p, int n, __int128 d) {
  if (d >= p.span[n] || -d >= p.span[n]) return false;
  if (n == 0) return true;
  const __int128 s = p.stride[n - 1], most = p.count[n - 1] - 1;
  const __int128 c = d >= 0 ? d / s : -((-d + s - 1) / s);  // d lies between c and c + 1 parts
  for (const __int128 x : {c, c + 1})
    if (x >= -most && x <= most && shifted_places_meet(p, n - 1, d - x * s)) return true;
  return false;
}

// n rows of `width` 2-byte elements, `stride` elements apart: some byte is the cache's (K or V).
bool rows_in_cache(const psispec_paged_cache* c, const void* rows, int64_t stride, int64_t width, int64_t n) {
  const Places p = cache_places(c);
  for (const void* base : {c->k, c->v}) {
    const __int128 at = (__int128)(uintptr_t)rows - (__int128)(uintptr_t)base;
    if (!bytes_in_places(p, p.levels, at, at + 2 * ((__int128)stride * (n - 1) + width))) continue;
    if (stride == width) return true;
    for (int64_t i = 0; i < n; ++i) {  // places in the rows' range, perhaps between the rows: rare
      const __int128 lo = at + 2 * (__int128)stride * i;
      if (bytes_in_places(p, p.levels, lo, lo + 2 * width)) return true;
    }
  }
  return false;
}

// n rows of wa elements, sa apart, and n of wb, sb apart: some element is in both.  Rows of equal stride
// may lie between each other (two parts of one packed projection).
bool rows_overlap(const void* a, int64_t sa, int64_t wa, const void* b, int64_t sb, int64_t wb, int64_t n) {
  const __int128 d = ((__int128)(uintptr_t)b - (__int128)(uintptr_t)a) / 2;
  if (d >= (__int128)sa * (n - 1) + wa || -d >= (__int128)sb * (n - 1) + wb) return false;
  if (sa == sb) {
    const int64_t m = (int64_t)((d % sa + sa) % sa);
    return m < wa || sa - m < wb;
  }
  for (int64_t i = 0, j = 0; i < n && j < n;) {  // one within the other: rare
    const __int128 at = (__int128)sa * i, bt = d + (__int128)sb * j;
    if (at + wa <= bt)
      ++i;
    else if (bt + wb <= at)
      ++j;
    else
      return true;
  }
  return false;
}

// The first na numbers at a and the first nb at b (either may be NULL): some number is in both.
bool ints_overlap(const int32_t* a, int64_t na, const int32_t* b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + 4 * (uintptr_t)nb && y < x + 4 * (uintptr_t)na;
}
// What a call reads of [batch] numbers lies apart from its status, which some workgroups write while others
// still read.
bool status_apart(const int32_t* status, int64_t batch, std::initializer_list<const int32_t*> read) {
  for (const int32_t* x : read)
    if (ints_overlap(status, batch, x, batch)) return false;
  return true;
}
// numbers from the first to the last of a table
int64_t table_extent(int64_t batch, int64_t stride, int64_t slots) { return (batch - 1) * stride + slots; }

bool cache_pointers_ok(const psispec_paged_cache* c) {
  return c->k && c->v && c->table && aligned(c->k, 16) && aligned(c->v, 16);
}

// Rows of `width` contiguous elements, `stride` elements apart, read and written 16 bytes at a time.
bool rows_ok(const void* p, int64_t stride, int64_t width) {
  return p && aligned(p, 16) && stride >= width && stride % 8 == 0;
}

psispec_status check_pool(const psispec_page_pool* p) {
  if (!p || p->reserved != 0) return PSISPEC_EINVAL;
  if (p->planes < 1 || p->num_pages < 1 || p->page_size < 1 || p->page_size > kMaxPageSize)
    return PSISPEC_EINVAL;
  if (p->row_bytes < 16 || p->row_bytes % 16 || p->row_bytes > (int64_t(1) << 32) ||
      p->plane_stride % 16 || p->page_stride % 16 || p->plane_stride < 0 ||
      p->page_stride < p->page_size * p->row_bytes)
    return PSISPEC_EINVAL;
  return PSISPEC_OK;
}

bool slots_ok(int32_t slots, int64_t table_stride, int32_t page_size) {
  return slots >= 1 && table_stride >= slots && (int64_t)slots * page_size <= kMaxPositions;
}

}  // namespace

extern "C" {

psispec_status psispec_qkv_append(const psispec_paged_cache* c, const psispec_qkv_prep* p,
                                  const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                  const void* v, int64_t v_stride, psispec_dtype dtype,
                                  int32_t batch, int32_t blk, int32_t heads_q,
                                  const int32_t* positions, const int32_t* len,
                                  const int32_t* n_new, void* q_out, int64_t q_out_stride,
                                  int32_t* status, void* stream) {
  const psispec_status e = check_cache(c, dtype);
  if (e != PSISPEC_OK) return e;
  if (batch < 0 || blk < 1 || blk > kMaxAppendBlock || heads_q < 1 || heads_q > kMaxHeads || !p)
    return PSISPEC_EINVAL;
  if (!cache_places(c).apart) return PSISPEC_EINVAL;
  if (!(p->eps >= 0.0) || !isfinite((float)p->eps) || !isfinite((float)p->rope_scale) || p->rot < 0 ||
      p->rot > c->dim || p->rot % 16 || (p->flags & ~PSISPEC_ROPE_INTERLEAVED) ||
      (p->rot > 0 && !p->inv_freq) || !aligned(p->q_weight, 16) || !aligned(p->k_weight, 16))
    return PSISPEC_EINVAL;
  if (!grid_ok((int64_t)batch * blk)) return PSISPEC_EINVAL;
  if (batch == 0) return PSISPEC_OK;
  if (!cache_pointers_ok(c) || !len) return PSISPEC_EINVAL;
  const int64_t wq = (int64_t)heads_q * c->dim, wk = (int64_t)c->heads * c->dim;
  if (!rows_ok(q, q_stride, wq) || !rows_ok(k, k_stride, wk) || !rows_ok(v, v_stride, wk) ||
      !rows_ok(q_out, q_out_stride, wq))
    return PSISPEC_EINVAL;
  const int64_t rows = (int64_t)batch * blk;
  if (!(q_out == q && q_out_stride == q_stride) &&
      rows_overlap(q, q_stride, wq, q_out, q_out_stride, wq, rows))
    return PSISPEC_EINVAL;
  if (rows_overlap(k, k_stride, wk, q_out, q_out_stride, wq, rows) ||
      rows_overlap(v, v_stride, wk, q_out, q_out_stride, wq, rows) ||
      rows_in_cache(c, q_out, q_out_stride, wq, rows))
    return PSISPEC_EINVAL;
  if (!status_apart(status, batch, {len, n_new}) || ints_overlap(status, batch, positions, rows) ||
      ints_overlap(status, batch, c->table, table_extent(batch, c->table_stride, c->slots)))
    return PSISPEC_EINVAL;
  const Places places = cache_places(c);
  if (shifted_places_meet(places, places.levels, (__int128)(uintptr_t)c->v - (__int128)(uintptr_t)c->k))
    return PSISPEC_EINVAL;
  AppendArgs a{};
  a.c = *c;
  a.p = *p;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = q_out;
  a.q_out_stride = q_out_stride;
  a.positions = positions;
  a.len = len;
  a.n_new = n_new;
  a.status = status;
  a.batch = batch;
  a.blk = blk;
  a.heads_q = heads_q;
  return launch_qkv_append(a, dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? PSISPEC_OK
                                                                                    : PSISPEC_EHIP;
}

static bool attend_sizes_ok(int32_t batch, int32_t blk, int32_t heads_q, int32_t heads_kv,
                            int32_t dim) {
  return batch >= 0 && blk >= 1 && blk <= kMaxAttendBlock && heads_kv >= 1 && heads_q >= heads_kv &&
         heads_q <= kMaxHeads && heads_q % heads_kv == 0 && dim >= 16 && dim <= kMaxHeadDim &&
         dim % 16 == 0 && grid_ok(batch);  // a workgroup per line at most (masks, status)
}

// The units of work that the kernel's shares are cut from, at most: their product with the 2^14 parts of a
// share's border stays below 2^63.
static bool attend_units_ok(const psispec_paged_cache* c, int32_t batch, int32_t blk, int32_t heads_q) {
  const int64_t groups = (int64_t)blk * (heads_q / c->heads) / 16 + 1;
  const int64_t steps = (int64_t)c->slots * c->page_size / 32 + 4;
  return (__int128)batch * c->heads * groups * steps < (__int128)1 << 49;
}

size_t psispec_paged_attention_workspace(int32_t batch, int32_t blk, int32_t heads_q,
                                         int32_t heads_kv, int32_t dim) {
  if (!attend_sizes_ok(batch, blk, heads_q, heads_kv, dim)) return 0;
  return attend_workspace_bytes(batch, blk, heads_q, heads_kv, dim);
}

psispec_status psispec_paged_attention(const psispec_paged_cache* c, const void* q, int64_t q_stride,
                                       psispec_dtype dtype, int32_t batch, int32_t blk,
                                       int32_t heads_q, const int32_t* parent, const int32_t* len,
                                       const int32_t* n_new, double scale, void* out,
                                       int64_t out_stride, int32_t* status, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  const psispec_status e = check_cache(c, dtype);
  if (e != PSISPEC_OK) return e;
  if (!attend_sizes_ok(batch, blk, heads_q, c->heads, c->dim) || !attend_units_ok(c, batch, blk, heads_q) ||
      !isfinite((float)scale * kLog2e))
    return PSISPEC_EINVAL;
  if (batch == 0) return PSISPEC_OK;
  const int64_t wq = (int64_t)heads_q * c->dim;
  if (!cache_pointers_ok(c) || !len || !rows_ok(q, q_stride, wq) || !rows_ok(out, out_stride, wq) ||
      rows_overlap(q, q_stride, wq, out, out_stride, wq, (int64_t)batch * blk) ||
      rows_in_cache(c, out, out_stride, wq, (int64_t)batch * blk))
    return PSISPEC_EINVAL;
  if (!status_apart(status, batch, {len, n_new}) || ints_overlap(status, batch, parent, (int64_t)batch * blk) ||
      ints_overlap(status, batch, c->table, table_extent(batch, c->table_stride, c->slots)))
    return PSISPEC_EINVAL;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < attend_workspace_bytes(batch, blk, heads_q, c->heads, c->dim))
    return PSISPEC_EWORKSPACE;
  AttendArgs a{};
  a.c = *c;
  a.q = q;
  a.out = out;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.parent = parent;
  a.len = len;
  a.n_new = n_new;
  a.status = status;
  a.scale = (float)scale;
  a.batch = batch;
  a.blk = blk;
  a.heads_q = heads_q;
  return launch_attend(a, dtype, workspace, static_cast<hipStream_t>(stream)) == hipSuccess
             ? PSISPEC_OK
             : PSISPEC_EHIP;
}

psispec_status psispec_paged_commit(const psispec_page_pool* pool, const int32_t* table,
                                    int64_t table_stride, int32_t slots, int32_t batch, int32_t blk,
                                    const int32_t* keep, int32_t keep_stride, const int32_t* n_keep,
                                    const int32_t* len, int32_t* new_len, int32_t* status,
                                    void* stream) {
  const psispec_status e = check_pool(pool);
  if (e != PSISPEC_OK) return e;
  if (batch < 0 || blk < 1 || blk > kMaxKvBlock || !slots_ok(slots, table_stride, pool->page_size) ||
      blk > (int64_t)slots * pool->page_size || (keep && keep_stride < 1))
    return PSISPEC_EINVAL;
  const int64_t tiles = pool->row_bytes / 16 > (int64_t(1) << 32) / pool->planes
                            ? INT64_C(1) << 32
                            : pool->planes * (pool->row_bytes / 16) / 256 + 1;
  if (!grid_ok(tiles) || !grid_ok(batch * tiles)) return PSISPEC_EINVAL;
  if (batch == 0) return PSISPEC_OK;
  if (!pool->base || !aligned(pool->base, 16) || !table || !n_keep || !len || !new_len)
    return PSISPEC_EINVAL;
  if (new_len != len && ints_overlap(new_len, batch, len, batch)) return PSISPEC_EINVAL;
  if (ints_overlap(new_len, batch, n_keep, batch) ||
      ints_overlap(new_len, batch, keep, (int64_t)batch * keep_stride) ||
      ints_overlap(new_len, batch, table, table_extent(batch, table_stride, slots)))
    return PSISPEC_EINVAL;
  if (!status_apart(status, batch, {len, n_keep, new_len}) ||
      ints_overlap(status, batch, keep, (int64_t)batch * keep_stride) ||
      ints_overlap(status, batch, table, table_extent(batch, table_stride, slots)))
    return PSISPEC_EINVAL;
  PagedCommitArgs a{};
  a.pool = *pool;
  a.table = table;
  a.table_stride = table_stride;
  a.slots = slots;
  a.batch = batch;
  a.blk = blk;
  a.keep = keep;
  a.keep_stride = keep_stride;
  a.n_keep = n_keep;
  a.len = len;
  a.new_len = new_len;
  a.status = status;
  return launch_paged_commit(a, static_cast<hipStream_t>(stream)) == hipSuccess ? PSISPEC_OK
                                                                               : PSISPEC_EHIP;
}

static size_t pages_ws(int32_t batch, int32_t slots, int32_t num_pages, int32_t blk,
                       int32_t page_size) {
  if (batch < 0 || batch > (1 << 23) || slots < 1 || num_pages < 1 || blk < 1 ||
      blk > kMaxAppendBlock || page_size < 1 || page_size > kMaxPageSize ||
      (int64_t)slots * page_size > kMaxPositions)
    return 0;
  return pages_workspace_bytes(batch, slots, num_pages, blk, page_size);
}

size_t psispec_pages_workspace(int32_t batch, int32_t slots, int32_t num_pages, int32_t blk,
                               int32_t page_size) {
  return pages_ws(batch, slots, num_pages, blk, page_size);
}

psispec_status psispec_pages_assign(int32_t* table, int64_t table_stride, int32_t slots,
                                    int32_t* refs, int32_t num_pages, int32_t page_size,
                                    int32_t* len, const int32_t* src, const int32_t* new_len,
                                    int32_t* status, int32_t batch, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  const size_t need = pages_ws(batch, slots, num_pages, 1, page_size);
  if (need == 0 || table_stride < slots) return PSISPEC_EINVAL;
  if (batch == 0) return PSISPEC_OK;
  if (!table || !refs || !len || !src || !new_len) return PSISPEC_EINVAL;
  if (!status_apart(status, batch, {len, src, new_len}) || ints_overlap(status, batch, refs, num_pages) ||
      ints_overlap(status, batch, table, table_extent(batch, table_stride, slots)))
    return PSISPEC_EINVAL;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return PSISPEC_EWORKSPACE;
  AssignArgs a{};
  a.table = table;
  a.table_stride = table_stride;
  a.slots = slots;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.batch = batch;
  a.refs = refs;
  a.len = len;
  a.src = src;
  a.new_len = new_len;
  a.status = status;
  return launch_pages_assign(a, workspace, static_cast<hipStream_t>(stream)) == hipSuccess
             ? PSISPEC_OK
             : PSISPEC_EHIP;
}

psispec_status psispec_pages_reserve(const psispec_page_pool* pool, int32_t* table,
                                     int64_t table_stride, int32_t slots, int32_t* refs,
                                     const int32_t* len, const int32_t* n_new, int32_t blk,
                                     int32_t* status, int32_t batch, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  const psispec_status e = check_pool(pool);
  if (e != PSISPEC_OK) return e;
  if (!slots_ok(slots, table_stride, pool->page_size)) return PSISPEC_EINVAL;
  const size_t need = pages_ws(batch, slots, pool->num_pages, blk, pool->page_size);
  if (need == 0) return PSISPEC_EINVAL;
  const int64_t per_plane = pool->page_size * pool->row_bytes / 16384 + 1;
  if (!grid_ok(per_plane) || !grid_ok(per_plane * pool->planes) ||
      !grid_ok(batch * (per_plane * pool->planes)))
    return PSISPEC_EINVAL;
  if (batch == 0) return PSISPEC_OK;
  if (!pool->base || !aligned(pool->base, 16) || !table || !refs || !len) return PSISPEC_EINVAL;
  if (!status_apart(status, batch, {len, n_new}) || ints_overlap(status, batch, refs, pool->num_pages) ||
      ints_overlap(status, batch, table, table_extent(batch, table_stride, slots)))
    return PSISPEC_EINVAL;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return PSISPEC_EWORKSPACE;
  ReserveArgs a{};
  a.pool = *pool;
  a.table = table;
  a.table_stride = table_stride;
  a.slots = slots;
  a.blk = blk;
  a.batch = batch;
  a.refs = refs;
  a.len = len;
  a.n_new = n_new;
  a.status = status;
  return launch_pages_reserve(a, workspace, static_cast<hipStream_t>(stream)) == hipSuccess
             ? PSISPEC_OK
             : PSISPEC_EHIP;
}

}  // extern "C"
