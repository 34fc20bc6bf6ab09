// w4_pack.hip -- weights of 4 bits, as a checkpoint holds them, into the order in which the products read
// them (layers.h, W4Layout).  Run once per layer when it is loaded: one wave per tile of 16 outputs x 128
// inputs, bytes read one at a time so that rows may start anywhere.
#include "layers.h"

namespace psispec {
namespace {

__global__ __launch_bounds__(256) void k_w4_pack(W4PackArgs a, W4Layout l) {
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (tile >= (int64_t)l.ntiles * l.ktiles) return;
  const int nt = (int)(tile / l.ktiles), t = (int)(tile - (int64_t)nt * l.ktiles);
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int n = nt * 16 + (lane & 15);
  const bool in = n < a.n;
  const bool mx = a.format == PSISPEC_W4_MX;
  const uint8_t* row = a.codes + (int64_t)n * a.codes_stride;
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = t * 128 + (mx ? 32 * g + 8 * j : 32 * j + 8 * g);
    uint32_t v = 0;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t b = in && k < a.k ? row[k / 2 + s] : 0;
      if (mx)
        v |= b << (8 * s);
      else
        v |= ((b & 15) << (4 * s)) | ((b >> 4) << (16 + 4 * s));
    }
    v ^= mx ? 0u : 0x88888888u;
    w[j] = mx ? v : v << 3 | v >> 29;
  }
  *reinterpret_cast<u32x4*>(a.packed + tile * 1024 + lane * 16) = u32x4{w[0], w[1], w[2], w[3]};
  if (mx) {
    const uint8_t* sc = static_cast<const uint8_t*>(a.scales) + (int64_t)n * a.scales_stride;
    const int blocks = a.k / 32, b = 4 * t + g;
    uint8_t* at = a.packed + l.scales_at + mx_scale_at(nt, t, l.ktiles) + 2 * lane;
    at[0] = in && b < blocks ? sc[b] : 0;
    if (t == l.ktiles - 1 && t % 2 == 0) at[1] = 0;  // no tile: never decoded but with rows of zeros
    if (t == 0) {
      int top = 0;
      if (in)
        for (int i = g; i < blocks; i += 4) top = max(top, (int)sc[i]);
      top = max(top, __shfl_xor(top, 16, 64));
      top = max(top, __shfl_xor(top, 32, 64));
      if (g == 0) a.packed[l.top_at + nt * 16 + lane] = (uint8_t)top;
    }
  } else if (g < l.gpt) {
    const uint16_t* sc = static_cast<const uint16_t*>(a.scales) + (int64_t)n * a.scales_stride;
    const int k = t * 128 + g * (128 / l.gpt);
    reinterpret_cast<uint16_t*>(a.packed + l.scales_at)[(tile * l.gpt + g) * 16 + (lane & 15)] =
        in && k < a.k ? sc[k / a.group] : 0;
  }
}

}  // namespace

hipError_t launch_w4_pack(const W4PackArgs& a, hipStream_t stream) {
  const W4Layout l = w4_layout(a.n, a.k, a.group, a.format);
  const int64_t tiles = (int64_t)l.ntiles * l.ktiles;
  PSISPEC_LAUNCH("w4_pack", k_w4_pack, dim3((unsigned)((tiles + 3) / 4)), dim3(256), 0, stream, a, l);
  return hipGetLastError();
}

}  // namespace psispec
