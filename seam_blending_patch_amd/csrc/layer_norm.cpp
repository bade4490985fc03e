// layer_norm.cpp -- host side of layer_norm_forward and layer_norm_backward:
// argument checks, the launch arguments and the workspace's layout.  No device
// memory is allocated and the stream is never synchronised.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "sb_host.h"
#include "sb_strided.h"
#include "sb_transformer.h"

using sb::failf;

namespace {

constexpr int64_t kMaxWidth = (int64_t)1 << 28; // D: element indices of a row are 32-bit

int read_shape(const int64_t *shape, sb::LNArgs &a) {
  if (!shape) return failf(SB_EARG, "null shape");
  const int64_t o = shape[0], i = shape[1], d = shape[2];
  if (o < 0 || i < 0 || d < 1) return failf(SB_EARG, "row counts must be >= 0 and the row length >= 1");
  if (o >= sb::kMaxExtent || i >= sb::kMaxExtent || o * i >= sb::kMaxExtent)
    return failf(SB_EGEOM, "2^31 rows or more");
  if (d > kMaxWidth) return failf(SB_EGEOM, "rows longer than 2^28 elements");
  std::memset(&a, 0, sizeof a);
  a.rows = o * i;
  a.inner = sb::make_fastdiv((uint32_t)std::max<int64_t>(i, 1));
  a.D = (int32_t)d;
  a.inv_d = 1.0f / (float)d;
  return SB_OK;
}

// checks one tensor's pointer and strides and describes it
int read_rows(const char *name, const void *p, const int64_t *stride, const int64_t *shape, int dtype,
              sb::RowStride &out, sb::Strided &s) {
  if (!p || !stride) return failf(SB_EARG, "null %s or strides of %s", name, name);
  for (int k = 0; k < 2; ++k)
    if (stride[k] < 0 || stride[k] >= sb::kMaxStride)
      return failf(SB_EGEOM, "strides of %s must be in 0..2^40 elements", name);
  if (!sb::aligned(p, sb::elem_bytes(dtype))) return failf(SB_EARG, "%s is not aligned to its element size", name);
  s.run = shape[2];
  s.add(shape[0], stride[0]);
  s.add(shape[1], stride[1]);
  if (s.span() >= sb::kMaxSpan) return failf(SB_EGEOM, "%s spans 2^52 elements or more", name);
  out = sb::RowStride{stride[0], stride[1]};
  return SB_OK;
}

// an output has to hold every element once, and to be the input itself or
// share nothing with it
int check_output(const char *name, const void *out, const sb::Strided &so, const char *in_name, const void *in,
                 const sb::Strided &si, int dtype) {
  if (!so.distinct()) return failf(SB_EARG, "%s overlaps itself", name);
  if (out == in && so.same(si)) return SB_OK;
  const int64_t eb = sb::elem_bytes(dtype), bytes = (int64_t)((uintptr_t)out - (uintptr_t)in);
  if (bytes % eb == 0 && sb::can_overlap(si, so, bytes / eb))
    return failf(SB_EARG, "%s overlaps %s without being it", name, in_name);
  return SB_OK;
}

int check_types(int dtype, int wdtype, const void *const *weights, int n) {
  if (!sb::known_dtype(dtype)) return failf(SB_EARG, "unknown dtype %d", dtype);
  if (wdtype != dtype && wdtype != SB_F32)
    return failf(SB_EARG, "weights must be of the rows' dtype or fp32 (got %d)", wdtype);
  for (int k = 0; k < n; ++k)
    if (weights[k] && !sb::aligned(weights[k], sb::elem_bytes(wdtype)))
      return failf(SB_EARG, "gamma, beta and their gradients must be aligned to their element size");
  return SB_OK;
}

// Stores pass the caches where the output alone fills the last-level one; below
// that, an operator that reads the rows next finds them there.  us with the hint
// and without, a call alone and (with such a reader behind it), rows of 2048 fp16:
//   output    forward                       backward
//    64 MB    25.4 /  32.2 ( 56 /  51)       47.5 /  48.9 ( 73 /  73)
//   128 MB    50.9 /  53.8 (100 / 101)       83.0 /  85.4 (137 / 134)
//   256 MB    94.9 /  99.0 (190 / 188)      156   / 159   (257 / 249)
//   512 MB   184   / 191   (364 / 363)      303   / 309   (489 / 484)
//     1 GB   365   / 375   (715 / 718)      605   / 621   (966 / 967)
bool past_caches(const sb::LNArgs &a, int dtype) {
  return a.rows * (int64_t)a.D * sb::elem_bytes(dtype) >= sb::kLastLevelBytes;
}

int check_eps(float eps) {
  return !(eps >= 0.0f) || eps == __builtin_inff() ? failf(SB_EARG, "eps must be finite and >= 0") : SB_OK;
}

// workspace of rows too long for registers: 8 floats a row and 8 a chunk of it
int64_t split_bytes(int64_t rows, int64_t d, int dtype, int64_t most) {
  const int64_t v = 16 / sb::elem_bytes(dtype), chunk = sb::kLNThreads * sb::kChunkVectors * v;
  return (d + v - 1) / v <= most ? 0 : rows * (1 + (d + chunk - 1) / chunk) * 8 * (int64_t)sizeof(float);
}

// The backward pass's workspace: nparts blocks of 2 * cols floats, then
// split_bytes.
struct BackwardPlan {
  int64_t nparts, cols, part_bytes, rowstat_bytes;
  int64_t blocks; // of a call that forms no weight gradients, and so no partials
};

int check_workspace(const void *workspace, size_t bytes, int64_t need) {
  if (need > 0 && (!workspace || !sb::aligned(workspace, 16)))
    return failf(SB_EARG, "workspace must be 16-byte aligned device memory");
  if (need > 0 && bytes < (size_t)need)
    return failf(SB_EWORKSPACE, "workspace too small: %zu bytes given, %lld needed", bytes, (long long)need);
  return SB_OK;
}

BackwardPlan plan_backward(int64_t rows, int64_t d, int dtype) {
  BackwardPlan p;
  const int64_t v = 16 / sb::elem_bytes(dtype), nv = (d + v - 1) / v;
  const sb::LNLayout lay = sb::backward_layout(nv);
  if (lay.lanes) {
    p.cols = (int64_t)lay.lanes * lay.nv * v;
    const int64_t blocks = (int64_t)sb_cu_count() * lay.blocks_per_cu();
    // Where there are weights' gradients to sum, a single block, whose sums need
    // no second launch, for what it can take in four turns and 2048 vectors: that
    // launch costs the host 3 to 4 us of a call of 11.  Kernels in us, one block
    // and several with the second launch, bf16: 16 rows of 768 7.8 / 6.7, 8 and
    // 16 of 2048 8.5 / 8.2 and 11.6 / 8.2, 8 of 4096 15 / 10.1, 2 of 8192 12.7 /
    // 10.8; past the rule 3 of 8192 14.7 / 10.8, 2 and 4 of 16384 21.5 / 14.7 and
    // 27.3 / 14.7, 32 of 2048 15 / 9.4.
    const int64_t turns = (rows + lay.rows() - 1) / lay.rows();
    p.blocks = std::min(turns, blocks);
    p.nparts = turns == 1 || (turns <= 4 && turns * nv <= 2048) ? 1 : p.blocks;
  } else {
    const int64_t per = sb::kLNThreads * v;
    p.cols = (d + per - 1) / per * per;
    p.nparts = std::max<int64_t>(1, std::min<int64_t>(rows, 4 * sb_cu_count() / std::max<int64_t>(1, p.cols / per)));
    p.blocks = p.nparts;
  }
  p.rowstat_bytes = split_bytes(rows, d, dtype, sb::kBackwardVectors);
  p.part_bytes = p.nparts * 2 * p.cols * (int64_t)sizeof(float);
  return p;
}

} // namespace

extern "C" size_t layer_norm_forward_workspace_bytes(const int64_t shape[3], int dtype) {
  sb::LNArgs a;
  if (!sb::known_dtype(dtype)) {
    failf(SB_EARG, "unknown dtype %d", dtype);
    return (size_t)-1;
  }
  if (read_shape(shape, a)) return (size_t)-1;
  return (size_t)split_bytes(a.rows, a.D, dtype, sb::kForwardVectors);
}

extern "C" int layer_norm_forward(const void *x, const int64_t x_stride[2], const int64_t shape[3], float eps,
                                  const void *gamma, const void *beta, int dtype, int weight_dtype, void *out,
                                  const int64_t out_stride[2], void *workspace, size_t workspace_bytes,
                                  void *stream) {
  sb::LNArgs a;
  int rc;
  const void *weights[2] = {gamma, beta};
  if ((rc = check_types(dtype, weight_dtype, weights, 2)) || (rc = read_shape(shape, a)) || (rc = check_eps(eps)))
    return rc;
  if (a.rows == 0) return SB_OK;
  sb::Strided sx, so;
  if ((rc = read_rows("x", x, x_stride, shape, dtype, a.sx, sx)) ||
      (rc = read_rows("out", out, out_stride, shape, dtype, a.sout, so)) ||
      (rc = check_output("out", out, so, "x", x, sx, dtype)))
    return rc;
  if ((rc = check_workspace(workspace, workspace_bytes, split_bytes(a.rows, a.D, dtype, sb::kForwardVectors))))
    return rc;
  a.rowstat = (float *)workspace;
  a.chunks = a.rowstat + a.rows * 8;
  a.x = x;
  a.out = out;
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.far = past_caches(a, dtype);
  const hipError_t e = sb_launch_layer_norm(a, dtype, weight_dtype, (hipStream_t)stream);
  if (e != hipSuccess) return failf(SB_ELAUNCH, "layer norm launch failed: %s", hipGetErrorString(e));
  return SB_OK;
}

extern "C" size_t layer_norm_backward_workspace_bytes(const int64_t shape[3], int dtype) {
  sb::LNArgs a;
  if (!sb::known_dtype(dtype)) {
    failf(SB_EARG, "unknown dtype %d", dtype);
    return 0;
  }
  if (read_shape(shape, a)) return 0;
  const BackwardPlan p = plan_backward(a.rows, a.D, dtype);
  return (size_t)(p.part_bytes + p.rowstat_bytes);
}

extern "C" int layer_norm_backward(const void *dy, const int64_t dy_stride[2], const void *x,
                                   const int64_t x_stride[2], const int64_t shape[3], float eps, const void *gamma,
                                   int dtype, int weight_dtype, void *dx, const int64_t dx_stride[2], void *dgamma,
                                   void *dbeta, void *workspace, size_t workspace_bytes, void *stream) {
  sb::LNArgs a;
  int rc;
  const void *weights[3] = {gamma, dgamma, dbeta};
  if ((rc = check_types(dtype, weight_dtype, weights, 3)) || (rc = read_shape(shape, a)) || (rc = check_eps(eps)))
    return rc;
  const bool wanted = dgamma || dbeta;
  if (a.rows == 0 && !wanted) return SB_OK;
  if (a.rows > 0) {
    sb::Strided sx, sdy, so;
    if ((rc = read_rows("dy", dy, dy_stride, shape, dtype, a.sdy, sdy)) ||
        (rc = read_rows("x", x, x_stride, shape, dtype, a.sx, sx)) ||
        (rc = read_rows("dx", dx, dx_stride, shape, dtype, a.sout, so)) ||
        (rc = check_output("dx", dx, so, "x", x, sx, dtype)) ||
        (rc = check_output("dx", dx, so, "dy", dy, sdy, dtype)))
      return rc;
  }
  const BackwardPlan p = plan_backward(a.rows, a.D, dtype);
  if ((rc = check_workspace(workspace, workspace_bytes, p.part_bytes + p.rowstat_bytes))) return rc;
  a.x = x;
  a.dy = dy;
  a.out = dx;
  a.gamma = gamma;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.eps = eps;
  a.far = past_caches(a, dtype);
  a.part = wanted ? (float *)workspace : nullptr;
  a.rowstat = (float *)((char *)workspace + p.part_bytes);
  a.chunks = a.rowstat + a.rows * 8;
  a.nparts = a.rows > 0 ? (int32_t)(wanted ? p.nparts : p.blocks) : 0;
  a.cols = (int32_t)p.cols;
  const hipError_t e = sb_launch_layer_norm_backward(a, dtype, weight_dtype, (hipStream_t)stream);
  if (e != hipSuccess) return failf(SB_ELAUNCH, "layer norm launch failed: %s", hipGetErrorString(e));
  return SB_OK;
}
