// paged.h -- launchers and device helpers of the paged KV cache: append, attention, pages.
#pragma once

#include "launch.h"

namespace psispec {

constexpr int kMaxPageSize = 4096;
constexpr int kMaxHeadDim = 256;
constexpr int kMaxAttendBlock = 1024;   // rows of a block that the attention takes
constexpr int kMaxAppendBlock = 1 << 20;
constexpr float kLog2e = 1.4426950408889634f;  // the scores are in powers of two

// append.hip
struct AppendArgs {
  psispec_paged_cache c;
  psispec_qkv_prep p;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements
  void* q_out;
  const int32_t *positions, *len, *n_new;
  int32_t* status;
  int batch, blk, heads_q;
};
hipError_t launch_qkv_append(const AppendArgs& a, psispec_dtype dtype, hipStream_t stream);

// attend.hip
struct AttendArgs {
  psispec_paged_cache c;
  const void* q;
  void* out;
  int64_t q_stride, out_stride;  // elements
  const int32_t *parent, *len, *n_new;
  int32_t* status;
  float scale;
  int batch, blk, heads_q;
};
size_t attend_workspace_bytes(int batch, int blk, int heads_q, int heads_kv, int dim);
hipError_t launch_attend(const AttendArgs& a, psispec_dtype dtype, void* workspace,
                         hipStream_t stream);

// pages.hip
struct PagedCommitArgs {
  psispec_page_pool pool;
  const int32_t* table;
  int64_t table_stride;
  int slots, batch, blk;
  const int32_t* keep;
  int keep_stride;
  const int32_t *n_keep, *len;
  int32_t *new_len, *status;
};
hipError_t launch_paged_commit(const PagedCommitArgs& a, hipStream_t stream);

struct AssignArgs {
  int32_t* table;
  int64_t table_stride;
  int slots, num_pages, page_size, batch;
  int32_t *refs, *len;
  const int32_t *src, *new_len;
  int32_t* status;
};
struct ReserveArgs {
  psispec_page_pool pool;
  int32_t* table;
  int64_t table_stride;
  int slots, blk, batch;
  int32_t* refs;
  const int32_t *len, *n_new;
  int32_t* status;
};
size_t pages_workspace_bytes(int batch, int slots, int num_pages, int blk, int page_size);
hipError_t launch_pages_assign(const AssignArgs& a, void* workspace, hipStream_t stream);
hipError_t launch_pages_reserve(const ReserveArgs& a, void* workspace, hipStream_t stream);

// New rows of line r and whether its lengths are valid: 0 <= len, 0 <= n <= blk and the rows fit
// the slots.
__device__ inline bool line_rows(const int32_t* len, const int32_t* n_new, int r, int blk, int slots,
                                 int page_size, int* L, int* n) {
  *L = len[r];
  *n = n_new ? n_new[r] : blk;
  return *L >= 0 && *n >= 0 && *n <= blk &&
         (int64_t)*L + *n <= (int64_t)slots * page_size;
}

}  // namespace psispec
