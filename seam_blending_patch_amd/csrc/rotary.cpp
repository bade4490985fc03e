// rotary.cpp -- host side of rotary_apply: argument checks and the launch
// arguments.  No device memory is allocated and the stream is never
// synchronised.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "sb_host.h"
#include "sb_strided.h"
#include "sb_transformer.h"

using sb::failf;

namespace {

constexpr int64_t kMaxHead = 1 << 13;  // head length: two tokens' cosines and sines are at most 64 KiB
constexpr int64_t kMaxHeads = 1 << 12; // heads of a tensor: steps of a token are 32-bit

int read_tensor(const char *name, const void *p, const int64_t stride[3], const int64_t shape[3], int64_t heads,
                int dtype, sb::Strided &s) {
  if (!p || !stride) return failf(SB_EARG, "null %s or strides of %s", name, name);
  for (int k = 0; k < 3; ++k)
    if (stride[k] < 0 || stride[k] >= sb::kMaxStride)
      return failf(SB_EGEOM, "strides of %s must be in 0..2^40 elements", name);
  if (!sb::aligned(p, sb::elem_bytes(dtype))) return failf(SB_EARG, "%s is not aligned to its element size", name);
  s.run = shape[2];
  s.add(shape[0], stride[0]);
  s.add(shape[1], stride[1]);
  s.add(heads, stride[2]);
  if (s.span() >= sb::kMaxSpan) return failf(SB_EGEOM, "%s spans 2^52 elements or more", name);
  return SB_OK;
}

bool overlap(const void *a, const sb::Strided &sa, const void *b, const sb::Strided &sb_, int dtype) {
  const int64_t eb = sb::elem_bytes(dtype), bytes = (int64_t)((uintptr_t)b - (uintptr_t)a);
  return bytes % eb != 0 || sb::can_overlap(sa, sb_, bytes / eb);
}

} // namespace

extern "C" int rotary_apply(const void *q, const int64_t q_stride[3], void *q_out, const int64_t q_out_stride[3],
                            int64_t q_heads, const void *k, const int64_t k_stride[3], void *k_out,
                            const int64_t k_out_stride[3], int64_t k_heads, const int64_t shape[3], int dtype,
                            const double *freqs, int64_t rot_dim, int layout, const void *positions,
                            int position_bytes, const int64_t position_stride[3], const int64_t *sections,
                            int n_sections, float scale, int transpose, void *stream) {
  if (!sb::known_dtype(dtype)) return failf(SB_EARG, "unknown dtype %d", dtype);
  if (!shape) return failf(SB_EARG, "null shape");
  if (layout != SB_ROTARY_HALF && layout != SB_ROTARY_INTERLEAVED) return failf(SB_EARG, "unknown layout %d", layout);
  const int64_t B = shape[0], T = shape[1], D = shape[2];
  if (B < 0 || T < 0 || q_heads < 0 || k_heads < 0) return failf(SB_EARG, "negative extent");
  if (D < 1 || D > kMaxHead) return failf(SB_EGEOM, "head length must be in 1..%lld", (long long)kMaxHead);
  if (q_heads > kMaxHeads || k_heads > kMaxHeads) return failf(SB_EGEOM, "more than %lld heads", (long long)kMaxHeads);
  if (B >= sb::kMaxExtent || T >= sb::kMaxExtent || B * T >= sb::kMaxExtent)
    return failf(SB_EGEOM, "2^31 tokens or more");
  if (rot_dim < 2 || rot_dim > D || rot_dim % 2 != 0)
    return failf(SB_EARG, "rot_dim must be even and in 2..%lld (got %lld)", (long long)D, (long long)rot_dim);
  if (position_bytes != 4 && position_bytes != 8) return failf(SB_EARG, "positions must be 4- or 8-byte integers");
  if (n_sections < 1 || n_sections > sb::kRotaryMaxAxes || !sections)
    return failf(SB_EARG, "1..%d sections of pairs", sb::kRotaryMaxAxes);
  if (!(scale > -__builtin_inff() && scale < __builtin_inff())) return failf(SB_EARG, "scale must be finite");

  sb::RotaryArgs a;
  std::memset(&a, 0, sizeof a);
  int64_t end = 0;
  for (int k2 = 0; k2 < n_sections; ++k2) {
    if (sections[k2] < 0 || sections[k2] > rot_dim) return failf(SB_EARG, "a section is negative or too long");
    end += sections[k2];
    a.ends[k2] = (int32_t)std::min<int64_t>(end, rot_dim);
  }
  if (end != rot_dim / 2)
    return failf(SB_EARG, "sections hold %lld pairs, the rotated part %lld", (long long)end, (long long)(rot_dim / 2));
  if (B * T == 0 || q_heads + k_heads == 0) return SB_OK;
  if (!freqs || !positions || !position_stride) return failf(SB_EARG, "null freqs, positions or their strides");
  if (!sb::aligned(freqs, 8) || !sb::aligned(positions, position_bytes))
    return failf(SB_EARG, "freqs and positions must be aligned to their element size");
  for (int k2 = 0; k2 < 3; ++k2)
    if (position_stride[k2] < 0 || position_stride[k2] >= sb::kMaxStride)
      return failf(SB_EGEOM, "strides of positions must be in 0..2^40 elements");
  sb::Strided sp;
  sp.run = 1;
  sp.add(n_sections, position_stride[0]);
  sp.add(B, position_stride[1]);
  sp.add(T, position_stride[2]);
  if (sp.span() >= sb::kMaxSpan) return failf(SB_EGEOM, "positions span 2^52 elements or more");

  const void *in[2] = {q, k};
  void *out[2] = {q_out, k_out};
  const int64_t *si[2] = {q_stride, k_stride}, *so[2] = {q_out_stride, k_out_stride}, heads[2] = {q_heads, k_heads};
  static const char *const kIn[2] = {"q", "k"}, *const kOut[2] = {"q_out", "k_out"};
  sb::Strided src[2], dst[2];
  int rc;
  for (int x = 0; x < 2; ++x) {
    if (heads[x] == 0) continue;
    if ((rc = read_tensor(kIn[x], in[x], si[x], shape, heads[x], dtype, src[x])) ||
        (rc = read_tensor(kOut[x], out[x], so[x], shape, heads[x], dtype, dst[x])))
      return rc;
    if (!dst[x].distinct()) return failf(SB_EARG, "%s overlaps itself", kOut[x]);
    a.x[x] = sb::RotaryTensor{in[x], out[x], si[x][0], si[x][1], si[x][2], so[x][0], so[x][1], so[x][2]};
    a.heads[x] = (int32_t)heads[x];
  }
  for (int x = 0; x < 2; ++x)
    for (int y = 0; y < 2; ++y) {
      if (heads[x] == 0 || heads[y] == 0) continue;
      const bool place = x == y && out[x] == in[y] && dst[x].same(src[y]);
      if (!place && overlap(in[y], src[y], out[x], dst[x], dtype))
        return failf(SB_EARG, "%s overlaps %s%s", kOut[x], kIn[y], x == y ? " without being it" : "");
      if (x < y && overlap(out[x], dst[x], out[y], dst[y], dtype)) return failf(SB_EARG, "q_out overlaps k_out");
    }

  const int64_t V = 16 / sb::elem_bytes(dtype);
  a.length = sb::make_fastdiv((uint32_t)T);
  a.D = (int32_t)D;
  a.part = (int32_t)rot_dim;
  const int64_t turned = layout == SB_ROTARY_INTERLEAVED ? rot_dim : rot_dim / 2;
  a.units_turned = (int32_t)((turned + V - 1) / V);
  a.units = a.units_turned + (int32_t)((D - rot_dim + V - 1) / V);
  a.items = a.units * (a.heads[0] + a.heads[1]);
  a.div_units = sb::make_fastdiv((uint32_t)a.units);
  a.div_items = sb::make_fastdiv((uint32_t)a.items);
  a.div_half = sb::make_fastdiv((uint32_t)(rot_dim / 2));
  a.freqs = freqs;
  a.positions = positions;
  a.pos_axis = position_stride[0];
  a.pos_b = position_stride[1];
  a.pos_t = position_stride[2];
  a.pos64 = position_bytes == 8;
  a.axes = n_sections;
  a.scale = scale;
  a.scale_sin = transpose ? -scale : scale;
  // launches of fewer than 2^31 steps: their indices are 32-bit
  const int64_t most = (((int64_t)1 << 31) - 1) / a.items;
  for (int64_t t0 = 0; t0 < B * T; t0 += most) {
    a.token0 = (uint32_t)t0;
    a.tokens = (uint32_t)std::min(most, B * T - t0);
    const hipError_t e = sb_launch_rotary(a, dtype, layout == SB_ROTARY_INTERLEAVED, (hipStream_t)stream);
    if (e != hipSuccess) return failf(SB_ELAUNCH, "rotary launch failed: %s", hipGetErrorString(e));
  }
  return SB_OK;
}
