// layers.h -- launchers of the layers around the paged attention: the norm with the residual's addition,
// linear layers with weights of 4 bits, the gated projections of a feed-forward block.
#pragma once

#include "launch.h"
#include "w4_plan.h"

namespace psispec {

// norm.hip
constexpr int kMaxNormDim = 32768;  // a row stays in the registers of one workgroup
enum NormOut { kNormSame = 0, kNormRow = 1, kNormMx = 2 };
struct AddNormArgs {
  const void *x, *residual, *weight;
  void *residual_out, *out, *scale;
  int64_t x_stride, residual_stride, residual_out_stride, out_stride, scale_stride;  // elements
  float eps;
  int rows, dim;
  int residual_f32;  // residual and residual_out hold 32-bit numbers, else x's type
  int kind;          // NormOut
};
hipError_t launch_add_rmsnorm(const AddNormArgs& a, psispec_dtype dtype, hipStream_t stream);

// Packed weights of 4 bits (w4_pack.hip).  Tiles of 16 outputs x 128 inputs; outputs and inputs behind
// the last have code 0 and scale 0.  Lane l of a wave (output l % 16, g = l / 16) owns the 16 bytes at
// 16 l of a tile, and word j of them holds its inputs
//   PSISPEC_W4_INT  32 j + 8 g + 0..7: nibble s, s + 4 = inputs 2s, 2s + 1 of the eight, code + 8; the word
//                   turned left by 3 bits
//   PSISPEC_W4_MX   32 g + 8 j + 0..7: nibble s = input s, the code as it is
// so word j is the lane's part of the j-th 16x16x32 matrix instruction of the tile (and the 16 bytes,
// for MX, its part of the 16x16x128 one).  Scales: INT [tile][groups per tile][16 outputs] in 16 bits,
// MX [tile of outputs][pair of tiles of inputs][64 lanes][2] a byte.  top (MX): the largest scale byte of each output.
struct W4Layout {
  int ntiles, ktiles, gpt;  // tiles of outputs, of inputs; groups per tile (INT; larger groups repeat)
  size_t scales_at, top_at, bytes;
};
inline W4Layout w4_layout(int n, int k, int group, int format) {
  W4Layout l{};
  l.ntiles = (n + 15) / 16;
  l.ktiles = (k + 127) / 128;
  l.gpt = group < 128 ? 128 / group : 1;
  const size_t tiles = (size_t)l.ntiles * l.ktiles;
  l.scales_at = tiles * 1024;
  l.top_at = l.scales_at + (format == PSISPEC_W4_MX ? (size_t)l.ntiles * ((l.ktiles + 1) / 2) * 128
                                                    : tiles * 32 * l.gpt);
  l.bytes = (l.top_at + (format == PSISPEC_W4_MX ? (size_t)l.ntiles * 16 : 0) + 255) / 256 * 256;
  return l;
}

// where the MX scale of lane 0 lies: tile t of the inputs of tile nt of the outputs; lane l's is 2 l further
__host__ __device__ inline int64_t mx_scale_at(int64_t nt, int t, int ktiles) {
  return (nt * ((ktiles + 1) / 2) + t / 2) * 128 + (t & 1);
}

struct W4PackArgs {
  const uint8_t* codes;
  const void* scales;
  int64_t codes_stride, scales_stride;  // bytes; elements
  uint8_t* packed;
  int n, k, group, format;
};
hipError_t launch_w4_pack(const W4PackArgs& a, hipStream_t stream);

// w4_*.hip
struct W4Args {
  const uint8_t* codes[2];  // the second of a gated call: the matrix that multiplies
  const void* scales[2];
  const uint8_t* top[2];
  int scale_f16;  // INT scales F16, else BF16
  const void* x;
  const uint8_t* x_scale;  // 8-bit rows: scale byte of every 32 inputs
  const void* bias;
  void* out;
  int64_t x_stride, xs_stride, out_stride;  // elements
  int rows, n, k, ntiles, ktiles, gpt;
  int act;      // psispec_w4_activation of a gated call
  int out_f16;  // out (and bias) F16, else BF16
  int out_vec;  // rows of out start at multiples of 8 bytes
  void* workspace;
};
hipError_t launch_w4_few_bf16(const W4Args& a, int format, int mats, hipStream_t stream);
hipError_t launch_w4_few_f16(const W4Args& a, int format, int mats, hipStream_t stream);
hipError_t launch_w4_few_f8(const W4Args& a, int mats, hipStream_t stream);
hipError_t launch_w4_many_bf16(const W4Args& a, int format, int mats, hipStream_t stream);
hipError_t launch_w4_many_f16(const W4Args& a, int format, int mats, hipStream_t stream);
hipError_t launch_w4_many_f8(const W4Args& a, int mats, hipStream_t stream);

size_t w4_workspace_bytes(int rows, int n, int k, int mats, int format);
hipError_t launch_w4(const W4Args& a, psispec_dtype dtype, int format, int mats, hipStream_t stream);

}  // namespace psispec
