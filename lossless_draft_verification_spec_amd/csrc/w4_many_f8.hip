// w4_many_f8.hip -- the 4-bit products of many rows for rows of 8 bits.
#include "w4_many.h"

namespace psispec {

size_t w4_many_workspace_bytes(int rows, int n, int k, int mats) {
  const size_t a = w4::many_plan(rows, n, k, mats, 1).bytes, b = w4::many_plan(rows, n, k, mats, 2).bytes;
  return a > b ? a : b;  // 16-bit and 8-bit rows
}
hipError_t launch_w4_many_f8(const W4Args& a, int mats, hipStream_t stream) {
  return mats == 2 ? w4::launch_many<w4::F8, 0, 2>(a, stream) : w4::launch_many<w4::F8, 0, 1>(a, stream);
}

}  // namespace psispec
