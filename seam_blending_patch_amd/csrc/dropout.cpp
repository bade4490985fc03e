// dropout.cpp -- host side of dropout_apply: argument checks and the launch
// arguments.  No device memory is allocated and the stream is never synchronised.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "sb_channels.h"
#include "sb_host.h"
#include "sb_strided.h"

using sb::failf;

namespace {

constexpr int64_t kMaxElements = (int64_t)1 << 34; // a counter of 32 bits for 4 elements each
constexpr int64_t kLaunchUnits = (int64_t)1 << 30;
constexpr int64_t kCaches = (int64_t)256 << 20;    // outputs that stores take past the caches

int read_rows(const char *name, const void *p, const int64_t *stride, const int64_t *shape, int dtype,
              int64_t (&out)[2], sb::Strided &s) {
  if (!p || !stride) return failf(SB_EARG, "null %s or strides of %s", name, name);
  for (int k = 0; k < 2; ++k)
    if (stride[k] < 0 || stride[k] >= sb::kMaxStride)
      return failf(SB_EGEOM, "strides of %s must be in 0..2^40 elements", name);
  if (!sb::aligned(p, sb::elem_bytes(dtype))) return failf(SB_EARG, "%s is not aligned to its element size", name);
  s.run = shape[2];
  s.add(shape[0], stride[0]);
  s.add(shape[1], stride[1]);
  if (s.span() >= sb::kMaxSpan) return failf(SB_EGEOM, "%s spans 2^52 elements or more", name);
  out[0] = stride[0];
  out[1] = stride[1];
  return SB_OK;
}

int check_apart(const void *out, const sb::Strided &so, const char *in_name, const void *in, const sb::Strided &si,
                int dtype) {
  if (out == in && so.same(si)) return SB_OK;
  const int64_t eb = sb::elem_bytes(dtype), bytes = (int64_t)((uintptr_t)out - (uintptr_t)in);
  if (bytes % eb != 0 || sb::can_overlap(si, so, bytes / eb))
    return failf(SB_EARG, "out overlaps %s without being it", in_name);
  return SB_OK;
}

} // namespace

extern "C" int dropout_apply(const void *x, const int64_t x_stride[2], const int64_t shape[3], int dtype, double p,
                             const int64_t *state, uint32_t site, const void *residual,
                             const int64_t residual_stride[2], void *out, const int64_t out_stride[2], void *stream) {
  if (!sb::known_dtype(dtype)) return failf(SB_EARG, "unknown dtype %d", dtype);
  if (!shape) return failf(SB_EARG, "null shape");
  const int64_t o = shape[0], i = shape[1], d = shape[2];
  if (o < 0 || i < 0 || d < 0) return failf(SB_EARG, "negative extent");
  if (!(p >= 0.0 && p < 1.0)) return failf(SB_EARG, "p must be in [0, 1)");
  if (o >= sb::kMaxExtent || i >= sb::kMaxExtent || o * i >= sb::kMaxExtent)
    return failf(SB_EGEOM, "2^31 rows or more");
  if (d > kMaxElements || (d > 0 && o * i > kMaxElements / d)) return failf(SB_EGEOM, "more than 2^34 elements");
  if (o * i == 0 || d == 0) return SB_OK;
  if (!state || !sb::aligned(state, 8)) return failf(SB_EARG, "state must be device memory of two 8-byte integers");

  sb::DropArgs a;
  std::memset(&a, 0, sizeof a);
  sb::Strided sx, sr, so;
  int rc;
  if ((rc = read_rows("x", x, x_stride, shape, dtype, a.sx, sx)) ||
      (residual && (rc = read_rows("residual", residual, residual_stride, shape, dtype, a.sr, sr))) ||
      (rc = read_rows("out", out, out_stride, shape, dtype, a.so, so)))
    return rc;
  if (!so.distinct()) return failf(SB_EARG, "out overlaps itself");
  if ((rc = check_apart(out, so, "x", x, sx, dtype)) ||
      (residual && (rc = check_apart(out, so, "residual", residual, sr, dtype))))
    return rc;
  a.x = x;
  a.residual = residual;
  a.out = out;
  a.D = d;
  a.inner = sb::make_fastdiv((uint32_t)i);
  a.state = state;
  a.site = site;
  a.threshold = (uint32_t)std::floor(p * 4294967296.0);
  a.scale = (float)(1.0 / (1.0 - p));
  a.quads = o * i == 1 || d % 4 == 0;
  a.far = o * i * d * sb::elem_bytes(dtype) >= kCaches;
  const int64_t v = 16 / sb::elem_bytes(dtype), units = (d + v - 1) / v, rows = o * i;
  const hipStream_t st = (hipStream_t)stream;
  hipError_t e = hipSuccess;
  if (units <= kLaunchUnits) { // whole rows, as many as a launch takes
    const int64_t most = kLaunchUnits / units;
    a.div_units = sb::make_fastdiv((uint32_t)units);
    for (int64_t r = 0; r < rows && e == hipSuccess; r += most) {
      a.row0 = r;
      a.units = (uint32_t)(std::min(most, rows - r) * units);
      e = sb_launch_dropout(a, dtype, st);
    }
  } else { // a row in pieces
    a.div_units = sb::make_fastdiv((uint32_t)kLaunchUnits);
    for (int64_t r = 0; r < rows; ++r)
      for (int64_t u = 0; u < units && e == hipSuccess; u += kLaunchUnits) {
        a.row0 = r;
        a.e0 = u * v;
        a.units = (uint32_t)std::min(kLaunchUnits, units - u);
        e = sb_launch_dropout(a, dtype, st);
      }
  }
  if (e != hipSuccess) return failf(SB_ELAUNCH, "dropout launch failed: %s", hipGetErrorString(e));
  return SB_OK;
}
