// layers_api.hip -- the C ABI of the layers around the paged attention: argument checks, then the launches of
// norm.hip, w4_pack.hip and w4.hip.
#include <math.h>

#include "layers.h"

using namespace psispec;

namespace {

constexpr int kMaxFeatures = 1 << 20;
constexpr int kMaxRows = (1 << 24) - 1;
constexpr int64_t kMaxTiles = (int64_t(1) << 26) - 4;  // of a weight: a wave each packs them, below 2^32 threads
constexpr int64_t kMaxStride = int64_t(1) << 36;  // elements: a row's offset stays below 2^62 bytes

constexpr int64_t kMaxRowStride = 1 << 24;  // bytes: 64 rows are reached by 32-bit offsets

bool aligned(const void* p, size_t n) { return (uintptr_t)p % n == 0; }

// `n` rows of `width` bytes, `stride` bytes apart
struct Rows {
  const void* p;
  int64_t stride, width, n;
};
__int128 reach(const Rows& r) { return (__int128)r.stride * (r.n - 1) + r.width; }

// Some byte is in a row of both.  Rows of equal stride may lie between each other (parts of one wider row).
bool meet(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.n < 1 || b.n < 1) return false;
  const __int128 d = (__int128)(uintptr_t)b.p - (__int128)(uintptr_t)a.p;
  if (d >= reach(a) || -d >= reach(b)) return false;
  if (a.stride == b.stride && a.n == b.n && a.stride > 0) {
    const int64_t m = (int64_t)((d % a.stride + a.stride) % a.stride);
    return m < a.width || a.stride - m < b.width;
  }
  for (int64_t i = 0, j = 0; i < a.n && j < b.n;) {  // one within the other: rare
    const __int128 at = (__int128)a.stride * i, bt = d + (__int128)b.stride * j;
    if (at + a.width <= bt)
      ++i;
    else if (bt + b.width <= at)
      ++j;
    else
      return true;
  }
  return false;
}
bool same(const Rows& a, const Rows& b) { return a.p == b.p && (a.n == 1 || a.stride == b.stride) && a.width == b.width; }

// A stride of rows that do not overlap; one row has none.
bool stride_ok(int64_t stride, int64_t width, int64_t rows) {
  return rows <= 1 || (stride >= width && stride <= kMaxStride);
}

int element_size(psispec_dtype t) { return t == PSISPEC_F32 ? 4 : t == PSISPEC_F8E4M3 || t == PSISPEC_E8M0 ? 1 : 2; }

psispec_status check_weight(const psispec_w4_weight* w) {
  if (!w || w->reserved != 0) return PSISPEC_EINVAL;
  if (w->n < 1 || w->n > kMaxFeatures || w->k < 32 || w->k > kMaxFeatures || w->k % 32) return PSISPEC_EINVAL;
  if ((int64_t)((w->n + 15) / 16) * ((w->k + 127) / 128) > kMaxTiles) return PSISPEC_EINVAL;
  if (w->format == PSISPEC_W4_MX) {
    if (w->group != 32) return PSISPEC_EINVAL;
    return w->scale_dtype == PSISPEC_E8M0 ? PSISPEC_OK : PSISPEC_EDTYPE;
  }
  if (w->format != PSISPEC_W4_INT) return PSISPEC_EUNSUPPORTED;
  if (w->group < 32 || w->group > kMaxFeatures || (w->group != 32 && w->group != 64 && w->group % 128))
    return PSISPEC_EINVAL;
  return w->scale_dtype == PSISPEC_BF16 || w->scale_dtype == PSISPEC_F16 ? PSISPEC_OK : PSISPEC_EDTYPE;
}

psispec_status check_packed(const psispec_w4_weight* w) {
  if (!w->packed || !aligned(w->packed, 256)) return PSISPEC_EINVAL;
  return PSISPEC_OK;
}

// What the two products share: rows of x, the scales of 8-bit rows, the output.
psispec_status product(const psispec_w4_weight* w, const psispec_w4_weight* w2, int act, const void* x,
                       int64_t x_stride, psispec_dtype dtype, const void* x_scale, int64_t xs_stride, int32_t rows,
                       const void* bias, void* out, int64_t out_stride, psispec_dtype out_dtype, void* workspace,
                       size_t workspace_bytes, void* stream) {
  psispec_status e = check_weight(w);
  if (e == PSISPEC_OK && w2) e = check_weight(w2);
  if (e != PSISPEC_OK) return e;
  if (dtype != PSISPEC_BF16 && dtype != PSISPEC_F16 && dtype != PSISPEC_F8E4M3) return PSISPEC_EDTYPE;
  const bool f8 = dtype == PSISPEC_F8E4M3;
  if (f8 ? out_dtype != PSISPEC_BF16 && out_dtype != PSISPEC_F16 : out_dtype != dtype) return PSISPEC_EDTYPE;
  if (f8 && w->format != PSISPEC_W4_MX) return PSISPEC_EUNSUPPORTED;
  if (w2 && (w2->n != w->n || w2->k != w->k || w2->group != w->group || w2->format != w->format ||
             w2->scale_dtype != w->scale_dtype)) return PSISPEC_EINVAL;
  if (rows < 0 || rows > kMaxRows) return PSISPEC_EINVAL;
  const int mats = w2 ? 2 : 1;
  const W4Layout l = w4_layout(w->n, w->k, w->group, w->format);
  // threads of a launch: below 2^32 (a workgroup of at most 512 per tile of 16 outputs and 16 rows)
  if ((int64_t)l.ntiles * ((rows + 15) / 16) > (int64_t(1) << 23) - 1) return PSISPEC_EINVAL;
  if (rows == 0) return PSISPEC_OK;
  if ((e = check_packed(w)) != PSISPEC_OK || (w2 && (e = check_packed(w2)) != PSISPEC_OK)) return e;
  const int xb = f8 ? 1 : 2;
  if (!x || !out || f8 != (x_scale != nullptr) || !aligned(x, 16) || !aligned(out, 2) || !aligned(bias, 2) || !stride_ok(x_stride, w->k, rows) ||
      (rows > 1 && (x_stride * xb % 16 || x_stride * xb > kMaxRowStride)) || !stride_ok(out_stride, w->n, rows) ||
      (f8 && !stride_ok(xs_stride, w->k / 32, rows)))
    return PSISPEC_EINVAL;
  const Rows ro{out, out_stride * 2, (int64_t)w->n * 2, rows}, rx{x, x_stride * xb, (int64_t)w->k * xb, rows},
      rs{x_scale, xs_stride, w->k / 32, rows}, rb{bias, 0, (int64_t)w->n * 2, 1},
      rw{w->packed, 0, (int64_t)l.bytes, 1}, rw2{w2 ? w2->packed : nullptr, 0, (int64_t)l.bytes, 1};
  if (meet(ro, rx) || meet(ro, rs) || meet(ro, rb) || meet(ro, rw) || meet(ro, rw2)) return PSISPEC_EINVAL;
  const size_t need = w4_workspace_bytes(rows, w->n, w->k, mats, w->format);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return PSISPEC_EWORKSPACE;
  const Rows rws{workspace, 0, (int64_t)need, need > 0};
  if (meet(rws, rx) || meet(rws, rs) || meet(rws, rb) || meet(rws, ro) || meet(rws, rw) || meet(rws, rw2))
    return PSISPEC_EINVAL;
  W4Args a{};
  for (int i = 0; i < mats; ++i) {
    const psispec_w4_weight* p = i ? w2 : w;
    a.codes[i] = static_cast<const uint8_t*>(p->packed);
    a.scales[i] = a.codes[i] + l.scales_at;
    a.top[i] = a.codes[i] + l.top_at;
  }
  a.scale_f16 = w->scale_dtype == PSISPEC_F16;
  a.x = x;
  a.x_scale = static_cast<const uint8_t*>(x_scale);
  a.bias = bias;
  a.out = out;
  a.x_stride = rows > 1 ? x_stride : 0;
  a.xs_stride = rows > 1 ? xs_stride : 0;
  a.out_stride = rows > 1 ? out_stride : 0;
  a.rows = rows;
  a.n = w->n;
  a.k = w->k;
  a.ntiles = l.ntiles;
  a.ktiles = l.ktiles;
  a.gpt = l.gpt;
  a.act = act;
  a.out_f16 = out_dtype == PSISPEC_F16;
  a.out_vec = aligned(out, 8) && a.out_stride % 4 == 0;
  a.workspace = workspace;
  return launch_w4(a, dtype, w->format, mats, static_cast<hipStream_t>(stream)) == hipSuccess ? PSISPEC_OK
                                                                                              : PSISPEC_EHIP;
}

}  // namespace

extern "C" {

psispec_status psispec_add_rmsnorm(const void* x, int64_t x_stride, psispec_dtype dtype, const void* residual,
                                   int64_t residual_stride, void* residual_out, int64_t residual_out_stride,
                                   psispec_dtype residual_dtype, const void* weight, double eps, int32_t rows,
                                   int32_t dim, void* out, int64_t out_stride, psispec_dtype out_dtype, void* scale,
                                   int64_t scale_stride, psispec_dtype scale_dtype, void* stream) {
  if (dtype != PSISPEC_BF16 && dtype != PSISPEC_F16) return PSISPEC_EDTYPE;
  if ((residual || residual_out) && residual_dtype != dtype && residual_dtype != PSISPEC_F32) return PSISPEC_EDTYPE;
  const bool quant = out_dtype == PSISPEC_F8E4M3;
  if (quant ? scale_dtype != PSISPEC_F32 && scale_dtype != PSISPEC_E8M0 : out_dtype != dtype) return PSISPEC_EDTYPE;
  const bool mx = quant && scale_dtype == PSISPEC_E8M0;
  if (rows < 0 || rows > kMaxRows || dim < 1 || dim > kMaxNormDim || (mx && dim % 32)) return PSISPEC_EINVAL;
  if (!(eps >= 0.0) || !isfinite((float)eps)) return PSISPEC_EINVAL;
  if (rows == 0) return PSISPEC_OK;
  const int rs = (residual || residual_out) && residual_dtype == PSISPEC_F32 ? 4 : 2;
  if (!x || !out || quant != (scale != nullptr) || !aligned(x, 2) || !aligned(weight, 2) || !aligned(residual, rs) ||
      !aligned(residual_out, rs) || !aligned(out, quant ? 1 : 2) || !aligned(scale, quant && !mx ? 4 : 1))
    return PSISPEC_EINVAL;
  if (!stride_ok(x_stride, dim, rows) || (residual && !stride_ok(residual_stride, dim, rows)) ||
      (residual_out && !stride_ok(residual_out_stride, dim, rows)) || !stride_ok(out_stride, dim, rows) ||
      (mx && !stride_ok(scale_stride, dim / 32, rows)))
    return PSISPEC_EINVAL;
  const Rows rx{x, x_stride * 2, (int64_t)dim * 2, rows}, rr{residual, residual_stride * rs, (int64_t)dim * rs, rows},
      rro{residual_out, residual_out_stride * rs, (int64_t)dim * rs, rows},
      ro{out, out_stride * element_size(out_dtype), (int64_t)dim * element_size(out_dtype), rows},
      rw{weight, 0, (int64_t)dim * 2, 1},
      rsc{scale, mx ? scale_stride : 4, mx ? dim / 32 : 4, quant ? rows : 0};
  // An output may be an input's rows themselves (a row is read whole before anything of it is written: each
  // thread writes what it has read); otherwise outputs lie apart from the inputs and from each other.
  const auto bad = [&](const Rows& w, const Rows& in) { return meet(w, in) && !same(w, in); };
  if (bad(ro, rx) || bad(ro, rr) || bad(rro, rx) || bad(rro, rr) || meet(ro, rro) || meet(ro, rw) || meet(rro, rw) ||
      meet(rsc, rx) || meet(rsc, rr) || meet(rsc, rro) || meet(rsc, ro) || meet(rsc, rw))
    return PSISPEC_EINVAL;
  AddNormArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.residual_out = residual_out;
  a.out = out;
  a.scale = scale;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.residual_out_stride = residual_out_stride;
  a.out_stride = out_stride;
  a.scale_stride = scale_stride;
  a.eps = (float)eps;
  a.rows = rows;
  a.dim = dim;
  a.residual_f32 = rs == 4;
  a.kind = !quant ? kNormSame : mx ? kNormMx : kNormRow;
  return launch_add_rmsnorm(a, dtype, static_cast<hipStream_t>(stream)) == hipSuccess ? PSISPEC_OK : PSISPEC_EHIP;
}

size_t psispec_w4_packed_bytes(int32_t n, int32_t k, int32_t group, int32_t format) {
  psispec_w4_weight w{};
  w.n = n;
  w.k = k;
  w.group = group;
  w.format = format;
  w.scale_dtype = format == PSISPEC_W4_MX ? PSISPEC_E8M0 : PSISPEC_BF16;
  return check_weight(&w) == PSISPEC_OK ? w4_layout(n, k, group, format).bytes : 0;
}

psispec_status psispec_w4_pack(const uint8_t* codes, int64_t codes_stride, const void* scales, int64_t scales_stride,
                               const psispec_w4_weight* w, size_t packed_bytes, void* stream) {
  psispec_status e = check_weight(w);
  if (e != PSISPEC_OK || (e = check_packed(w)) != PSISPEC_OK) return e;
  const W4Layout l = w4_layout(w->n, w->k, w->group, w->format);
  if (packed_bytes < l.bytes) return PSISPEC_EWORKSPACE;
  const int64_t groups = (w->k + w->group - 1) / w->group;
  const int ss = w->format == PSISPEC_W4_MX ? 1 : 2;
  if (!codes || !scales || !aligned(scales, ss) || !stride_ok(codes_stride, w->k / 2, w->n) ||
      !stride_ok(scales_stride, groups, w->n))
    return PSISPEC_EINVAL;
  const Rows rp{w->packed, 0, (int64_t)l.bytes, 1};
  if (meet(rp, Rows{codes, codes_stride, w->k / 2, w->n}) ||
      meet(rp, Rows{scales, scales_stride * ss, groups * ss, w->n}))
    return PSISPEC_EINVAL;
  W4PackArgs a{codes, scales, codes_stride, scales_stride, static_cast<uint8_t*>(w->packed),
               w->n, w->k, w->group, w->format};
  return launch_w4_pack(a, static_cast<hipStream_t>(stream)) == hipSuccess ? PSISPEC_OK : PSISPEC_EHIP;
}

size_t psispec_w4_workspace(int32_t rows, int32_t n, int32_t k, int32_t mats) {
  if (rows < 1 || rows > kMaxRows || n < 1 || n > kMaxFeatures || k < 32 || k > kMaxFeatures || mats < 1 || mats > 2)
    return 0;
  return w4_workspace_bytes(rows, n, k, mats, PSISPEC_W4_INT);
}

size_t psispec_w4_weight_workspace(const psispec_w4_weight* w, int32_t rows, int32_t mats) {
  if (check_weight(w) != PSISPEC_OK || rows < 1 || rows > kMaxRows || mats < 1 || mats > 2) return 0;
  return w4_workspace_bytes(rows, w->n, w->k, mats, w->format);
}

psispec_status psispec_w4_linear(const psispec_w4_weight* w, const void* x, int64_t x_stride, psispec_dtype dtype,
                                 const void* x_scale, int64_t x_scale_stride, int32_t rows, const void* bias, void* out,
                                 int64_t out_stride, psispec_dtype out_dtype, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  return product(w, nullptr, 0, x, x_stride, dtype, x_scale, x_scale_stride, rows, bias, out, out_stride, out_dtype,
                 workspace, workspace_bytes, stream);
}

psispec_status psispec_w4_gated(const psispec_w4_weight* gate, const psispec_w4_weight* up, int32_t activation,
                                const void* x, int64_t x_stride, psispec_dtype dtype, const void* x_scale,
                                int64_t x_scale_stride, int32_t rows, void* out, int64_t out_stride,
                                psispec_dtype out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!up || activation < PSISPEC_W4_SILU || activation > PSISPEC_W4_GELU_TANH) return PSISPEC_EINVAL;
  return product(gate, up, activation, x, x_stride, dtype, x_scale, x_scale_stride, rows, nullptr, out, out_stride,
                 out_dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
