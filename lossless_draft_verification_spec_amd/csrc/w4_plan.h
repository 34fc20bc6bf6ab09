// w4_plan.h -- which kernel takes a 4-bit product, and how the work is cut: rules on the sizes alone.  Host code
// without the GPU's headers.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "psispec.h"

namespace psispec {

// How the work of many rows is cut
struct ManyPlan {
  bool use;    // else the kernel for few rows takes it
  int nb;      // tiles of outputs of a wave, of all matrices
  int mblocks, nblocks, parts, mpad, npad;
  int band;    // row blocks that follow each other before the next column
  int steps;   // tiles of 128 inputs of a part, an even number
  size_t part_at, bytes;
};
// The kernel for many rows reads the weights once per 64 rows and the rows once per 256 outputs, the one for few
// rows in tiles of at most 64 x 64 whose waves share the inputs: that one where there are not tiles of 64 x 256
// enough for the CUs.  In us per launch, in a graph of 42 on three sets of inputs, few / many: 256 rows, 4096 x 4096
// (64 tiles) INT 16 / 45; 576 rows, 4096 x 4096 (144) INT 36.5 / 40.8; 256 rows, 12288 x 4096 (192) INT 38 / 41, MX
// 32.7 / 30.6, 8-bit rows 24 / 21; 576 rows, 6144 x 4096 (216) 8-bit rows 25.5 / 21.4.  Tiles of 64 x 128 up to 1.5
// tiles of 64 x 256 per CU (576 rows, 6144 x 4096: INT 41 against 46.5, MX 31.6 against 36.3; 12288 x 4096 MX: 55.2
// against 52.7).  Long rows with too few tiles: the inputs are cut so that there are about 432 workgroups (576 rows,
// 4096 x 12288: INT few 92, uncut 117, three parts 72; 8-bit rows 48, 56 and 39).
inline ManyPlan many_plan(int rows, int n, int k, int mats, int format) {
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

// How the work of few rows is cut.
struct FewPlan {
  int r4;  // rows of a workgroup over 4
  int nt;  // tiles of 16 outputs of a workgroup
  int kw;  // its waves
  int64_t blocks;
};
// The largest tile whose workgroups still cover most of the 256 CUs: a tile of twice the rows or outputs reads
// the weights or the rows once instead of twice.  In us as above: 64 rows, 4096 x 4096 INT: 64 rows x 64 outputs (64
// workgroups) 13.6, 32 x 64 (128) 9.9, 32 x 32 (256) 7.7, 16 x 32 (512) 8.4, 16 x 16 (1024) 10.4; 12288 x 4096: 64 x 64
// (192) 15.3, 32 x 64 (384) 15.9, 32 x 32 (768) 16.1.  Eight waves share a tile's inputs, four where several workgroups
// share a CU (64 rows, 24576 x 4096: INT 24.2 against 27.1, MX 20.7 against 24.4), sixteen for long rows (4096 x 12288:
// 9 rows 7.8 against 9.3, one row 7.5 against 9.3).  Little more than one workgroup per CU costs as much as two: 639
// rows, 2 x 208 x 9856 gated with 16 rows x 32 outputs (280 workgroups) 27.1, 32 x 32 (140) 21.3; 9 rows, 2 x 12288 x
// 4096 with 32 outputs (384) 13.5, 16 (768) 11.9, but 2 x 8192 and 2 x 24576 (256 and 768) 9.7 and 22.0 against 9.4 and
// 25.7.
inline FewPlan few_plan(int rows, int ntiles, int ktiles, int mats) {
  constexpr int kFill = 192, kShare = 320, kLong = 64;  // workgroups, workgroups, tiles of 128 inputs
  constexpr int kOne = 256, kTwo = 448;                 // workgroups: one, nearly two per CU
  const int wide = mats == 2 ? 2 : 4;
  const auto blocks = [&](int r4, int nt) {
    return (int64_t)((ntiles + nt - 1) / nt) * ((rows + 4 * r4 - 1) / (4 * r4));
  };
  const auto plan = [&](int r4, int nt, int kw) { return FewPlan{r4, nt, kw, blocks(r4, nt)}; };
  if (rows > 32 && blocks(16, wide) >= kFill) return plan(16, wide, blocks(16, wide) >= kShare ? 4 : 8);
  if (mats == 1 && rows > 16 && blocks(8, 4) >= kFill) return plan(8, 4, blocks(8, 4) >= kShare ? 4 : 8);
  if (rows > 16 && (blocks(8, 2) >= kFill || blocks(4, 2) > kOne)) return plan(8, 2, blocks(8, 2) >= kShare ? 4 : 8);
  if (rows > 4) {
    const int64_t b = blocks(4, 2);
    if ((b >= kFill && b <= kOne) || b >= kTwo) return plan(4, 2, 8);
    return plan(4, 1, ktiles >= kLong && b < kFill ? 16 : 8);
  }
  return plan(1, 1, ktiles >= kLong && blocks(1, 1) <= 256 ? 16 : 8);
}

}  // namespace psispec
