// w4.hip -- which kernel takes a 4-bit product, and how.
#include "layers.h"

namespace psispec {

// The kernel for many rows reads the weights once per 64 rows and the rows once per 256 outputs, the one for few
// rows in tiles of at most 64 x 64 whose waves share the inputs: that one where there are not tiles of 64 x 256
// enough for the CUs.  In us, few / many: 256 rows, 4096 x 4096 (64 tiles) INT 15.8 / 23.0; 576 rows, 4096 x
// 4096 (144) 32.8 / 36.7; 256 rows, 12288 x 4096 (192) INT 38 / 41, MX 33 / 31, 8-bit rows 25 / 21; 576 rows,
// 6144 x 4096 (216) 8-bit rows 25 / 21.  Tiles of 64 x 128 up to 1.5 tiles of 64 x 256 per CU (576 rows, 6144 x
// 4096: MX 31.8 against 36.0; 12288 x 4096: 57 against 53).  Long rows with too few tiles: the inputs are cut so
// that there are about 432 workgroups (576 rows, 4096 x 12288: INT few 85, three parts 75; 8-bit rows 48 / 39).
ManyPlan many_plan(int rows, int n, int k, int mats, int format) {
  constexpr int kRows = 64, kCus = 256;
  ManyPlan p{};
  const int ktiles = (k + 127) / 128, bn = 256 / mats;
  p.mblocks = (rows + kRows - 1) / kRows;
  p.nblocks = (n + bn - 1) / bn;
  p.mpad = p.mblocks * kRows;
  const int bands = p.mblocks < 12 ? 1 : (p.mblocks + 4) / 8;
  p.band = (p.mblocks + bands - 1) / bands;
  p.npad = (n + 15) / 16 * 16;
  const int64_t blocks = (int64_t)p.mblocks * p.nblocks;
  const bool cut = blocks >= kCus * 3 / 8 && ktiles >= 64;
  p.use = rows > kRows && (blocks >= kCus * 3 / 4 || cut);
  p.parts = 1;
  p.nb = 4;
  if (blocks < kCus * 3 / 4) {
    p.parts = (int)((432 + blocks / 2) / blocks);
  } else if (blocks < kCus * 3 / 2) {
    p.nb = 2;
    p.nblocks = (n + bn / 2 - 1) / (bn / 2);
  }
  p.steps = ((ktiles + p.parts - 1) / p.parts + 1) / 2 * 2;
  p.parts = (ktiles + p.steps - 1) / p.steps;
  // INT: the sums of up to four groups per tile
  p.part_at = format == PSISPEC_W4_INT ? ((size_t)ktiles * 4 * p.mpad * 4 + 255) / 256 * 256 : 0;
  p.bytes = p.part_at + (p.parts > 1 ? (size_t)p.parts * mats * rows * p.npad * 4 : 0);
  return p;
}

size_t w4_workspace_bytes(int rows, int n, int k, int mats, int format) {
  const ManyPlan p = many_plan(rows, n, k, mats, format);
  return p.use ? p.bytes : 0;
}

hipError_t launch_w4(const W4Args& a, psispec_dtype dtype, int format, int mats, hipStream_t stream) {
  const bool many = many_plan(a.rows, a.n, a.k, mats, format).use;
  if (dtype == PSISPEC_BF16)
    return many ? launch_w4_many_bf16(a, format, mats, stream) : launch_w4_few_bf16(a, format, mats, stream);
  if (dtype == PSISPEC_F16)
    return many ? launch_w4_many_f16(a, format, mats, stream) : launch_w4_few_f16(a, format, mats, stream);
  return many ? launch_w4_many_f8(a, mats, stream) : launch_w4_few_f8(a, mats, stream);
}

}  // namespace psispec
