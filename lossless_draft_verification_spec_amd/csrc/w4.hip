// w4.hip -- which kernel takes a 4-bit product.
#include "layers.h"

namespace psispec {

constexpr int kFewRows = 64;

size_t w4_workspace_bytes(int rows, int n, int k, int mats) {
  return rows <= kFewRows ? 0 : w4_many_workspace_bytes(rows, n, k, mats);
}

hipError_t launch_w4(const W4Args& a, psispec_dtype dtype, int format, int mats, hipStream_t stream) {
  // the kernel for many rows reaches 128 rows with 32-bit offsets
  const bool few = a.rows <= kFewRows || a.x_stride * (dtype == PSISPEC_F8E4M3 ? 1 : 2) > (1 << 30) / 128;
  if (dtype == PSISPEC_BF16)
    return few ? launch_w4_few_bf16(a, format, mats, stream) : launch_w4_many_bf16(a, format, mats, stream);
  if (dtype == PSISPEC_F16)
    return few ? launch_w4_few_f16(a, format, mats, stream) : launch_w4_many_f16(a, format, mats, stream);
  return few ? launch_w4_few_f8(a, mats, stream) : launch_w4_many_f8(a, mats, stream);
}

}  // namespace psispec
