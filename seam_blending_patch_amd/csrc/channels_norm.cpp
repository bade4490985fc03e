// channels_norm.cpp -- host side of group_norm_forward and group_norm_backward:
// argument checks, how positions are cut into blocks, the workspace's layout.  No
// device memory is allocated and the stream is never synchronised.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "sb_channels.h"
#include "sb_host.h"
#include "sb_strided.h"

using sb::failf;

namespace {

constexpr int64_t kMaxChannels = 1 << 16;
// samples times groups: a block of 1024 threads each, beside those for the channels,
// in a grid of fewer than 2^32 threads
constexpr int64_t kMaxGroups = (1 << 22) - (1 << 12);
constexpr int64_t kMaxPositions = (int64_t)1 << 30; // of a sample: a chunk's end is a 32-bit sum

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

int read_shape(const int64_t *shape, int64_t groups, int dtype, sb::ChanArgs &a) {
  if (!sb::known_dtype(dtype)) return failf(SB_EARG, "unknown dtype %d", dtype);
  if (!shape) return failf(SB_EARG, "null shape");
  const int64_t N = shape[0], S = shape[1], C = shape[2];
  if (N < 0 || S < 0 || C < 1) return failf(SB_EARG, "samples and positions must be >= 0, channels >= 1");
  if (groups < 1 || C % groups != 0)
    return failf(SB_EARG, "channels (%lld) must be a multiple of groups (%lld)", (long long)C, (long long)groups);
  if (C > kMaxChannels) return failf(SB_EGEOM, "more than %lld channels", (long long)kMaxChannels);
  if (S >= kMaxPositions || N >= sb::kMaxExtent || N * groups > kMaxGroups)
    return failf(SB_EGEOM, "2^30 positions of a sample or more, or more than 2^22 - 2^12 samples times groups");
  std::memset(&a, 0, sizeof a);
  a.N = (int32_t)N;
  a.S = (int32_t)S;
  a.C = (int32_t)C;
  a.G = (int32_t)groups;
  a.Cg = (int32_t)(C / groups);
  a.div_Cg = sb::make_fastdiv((uint32_t)a.Cg);
  const int64_t v = 16 / sb::elem_bytes(dtype);
  a.NV = (int32_t)((C + v - 1) / v);
  a.slabs = (a.NV + sb::kChanThreads - 1) / sb::kChanThreads;
  a.CV = (a.NV + a.slabs - 1) / a.slabs;
  a.RB = sb::kChanThreads / a.CV;
  a.div_CV = sb::make_fastdiv((uint32_t)a.CV);
  a.div_slabs = sb::make_fastdiv((uint32_t)a.slabs);
  // Blocks of the pass that sums: two a CU where each thread has 4 positions at
  // least, for each leaves partials that a merge reads (512 x 512 x 256 of two
  // samples fp16 with 2, 4 and 8 a CU: 164, 172 and 174 us in all; 256 x 256 x 512
  // bf16 backward 69, 76 and 93).
  const int64_t least = (int64_t)a.RB * 4, cus = sb_cu_count();
  const auto cut = [&](int64_t want, int32_t &chunk, int32_t &chunks) {
    const int64_t most = std::max<int64_t>(1, want / std::max<int64_t>(1, N * a.slabs));
    const int64_t n = std::max<int64_t>(1, std::min(most, (S + least - 1) / least));
    chunk = (int32_t)std::min<int64_t>(up((S + n - 1) / n, a.RB), sb::kMaxExtent - 1);
    chunks = chunk ? (int32_t)((S + chunk - 1) / chunk) : 0;
  };
  cut(2 * cus, a.chunk, a.chunks);
  cut(16 * cus, a.apply_chunk, a.apply_chunks); // (leaves none)
  a.div_chunks = sb::make_fastdiv((uint32_t)std::max(a.chunks, 1));
  a.far = N * S * C * sb::elem_bytes(dtype) >= (int64_t)256 << 20;
  return SB_OK;
}

// Groups for a block to hold: the fewest that fill whole vectors, where `vectors`
// of each of `threads` threads have room for their positions.  Then the merge's partials are one chunk
// of a sample (for the weights' gradients, which add up over samples).
void hold(sb::ChanArgs &a, int dtype, int64_t threads, int64_t vectors) {
  const int64_t v = 16 / sb::elem_bytes(dtype);
  int64_t sg = 1;
  while (sg <= v && sg * a.Cg % v != 0) ++sg;
  if (sg > v || a.G % sg != 0) return;
  const int64_t cv = sg * a.Cg / v;
  if (cv > threads || (a.S + threads / cv - 1) / (threads / cv) > vectors) return; // (positions of a turn, turns)
  a.sg = (int32_t)sg;
  a.CS = (int32_t)(sg * a.Cg);
  a.div_CVs = sb::make_fastdiv((uint32_t)cv);
  a.chunks = 1;
  a.chunk = a.S;
}

int read_positions(const char *name, const void *p, const int64_t *stride, const sb::ChanArgs &a, int dtype,
                   sb::SampleStride &out, sb::Strided &s) {
  if (!p || !stride) return failf(SB_EARG, "null %s or strides of %s", name, name);
  for (int k = 0; k < 2; ++k)
    if (stride[k] < 0 || stride[k] >= sb::kMaxStride)
      return failf(SB_EGEOM, "strides of %s must be in 0..2^40 elements", name);
  if (!sb::aligned(p, sb::elem_bytes(dtype))) return failf(SB_EARG, "%s is not aligned to its element size", name);
  s.run = a.C;
  s.add(a.N, stride[0]);
  s.add(a.S, stride[1]);
  if (s.span() >= sb::kMaxSpan) return failf(SB_EGEOM, "%s spans 2^52 elements or more", name);
  out = sb::SampleStride{stride[0], stride[1]};
  return SB_OK;
}

int check_output(const char *name, const void *out, const sb::Strided &so, const char *in_name, const void *in,
                 const sb::Strided &si, int dtype) {
  if (!so.distinct()) return failf(SB_EARG, "%s overlaps itself", name);
  if (out == in && so.same(si)) return SB_OK;
  const int64_t eb = sb::elem_bytes(dtype), bytes = (int64_t)((uintptr_t)out - (uintptr_t)in);
  if (bytes % eb != 0 || sb::can_overlap(si, so, bytes / eb))
    return failf(SB_EARG, "%s overlaps %s without being it", name, in_name);
  return SB_OK;
}

int check_types(int activation, int dtype, int wdtype, const void *const *weights, int n) {
  if (activation != SB_ACT_NONE && activation != SB_ACT_SILU) return failf(SB_EARG, "unknown activation %d", activation);
  if (wdtype != dtype && wdtype != SB_F32)
    return failf(SB_EARG, "weights must be of x's dtype or fp32 (got %d)", wdtype);
  for (int k = 0; k < n; ++k)
    if (weights[k] && !sb::aligned(weights[k], sb::elem_bytes(wdtype)))
      return failf(SB_EARG, "gamma, beta and their gradients must be aligned to their element size");
  return SB_OK;
}

// gradients of the weights are written while others are still read: none may share memory
int check_weights_apart(const void *const *weights, int wdtype, int64_t C) {
  static const char *const names[4] = {"gamma", "beta", "dgamma", "dbeta"};
  const uintptr_t bytes = (uintptr_t)C * sb::elem_bytes(wdtype);
  for (int x = 2; x < 4; ++x)
    for (int y = 0; y < x; ++y) {
      const uintptr_t a = (uintptr_t)weights[x], b = (uintptr_t)weights[y];
      if (a && b && a < b + bytes && b < a + bytes) return failf(SB_EARG, "%s overlaps %s", names[x], names[y]);
    }
  return SB_OK;
}

// floats: partials by chunk and channel (three forward, two backward), then the groups'
// statistics (or means)
int64_t part_floats(const sb::ChanArgs &a) { return up(3 * (int64_t)a.N * a.chunks * a.C, 4); }
int64_t workspace_bytes(const sb::ChanArgs &a) {
  return (part_floats(a) + up(3 * (int64_t)a.N * a.G, 4)) * (int64_t)sizeof(float);
}

int check_workspace(const void *workspace, size_t bytes, int64_t need) {
  if (need > 0 && (!workspace || !sb::aligned(workspace, 16)))
    return failf(SB_EARG, "workspace must be 16-byte aligned device memory");
  if (need > 0 && bytes < (size_t)need)
    return failf(SB_EWORKSPACE, "workspace too small: %zu bytes given, %lld needed", bytes, (long long)need);
  return SB_OK;
}

} // namespace

extern "C" size_t group_norm_workspace_bytes(const int64_t shape[3], int64_t groups, int dtype) {
  sb::ChanArgs a;
  if (read_shape(shape, groups, dtype, a)) return (size_t)-1;
  return (size_t)workspace_bytes(a);
}

extern "C" int group_norm_forward(const void *x, const int64_t x_stride[2], const int64_t shape[3], int64_t groups,
                                  float eps, const void *gamma, const void *beta, int activation, int dtype,
                                  int weight_dtype, void *out, const int64_t out_stride[2], float *stats,
                                  void *workspace, size_t workspace_bytes_, void *stream) {
  sb::ChanArgs a;
  int rc;
  const void *weights[2] = {gamma, beta};
  if ((rc = read_shape(shape, groups, dtype, a)) || (rc = check_types(activation, dtype, weight_dtype, weights, 2)))
    return rc;
  if (!(eps >= 0.0f) || eps == __builtin_inff()) return failf(SB_EARG, "eps must be finite and >= 0");
  if (!sb::aligned(stats, 4)) return failf(SB_EARG, "stats must be aligned to its element size");
  if (a.N == 0 || a.S == 0) return SB_OK;
  sb::Strided sx, so;
  if ((rc = read_positions("x", x, x_stride, a, dtype, a.sx, sx)) ||
      (rc = read_positions("out", out, out_stride, a, dtype, a.sout, so)) ||
      (rc = check_output("out", out, so, "x", x, sx, dtype)) ||
      (rc = check_workspace(workspace, workspace_bytes_, workspace_bytes(a))))
    return rc;
  a.x = x;
  a.out = out;
  a.gamma = gamma;
  a.beta = beta;
  a.silu = activation == SB_ACT_SILU;
  a.eps = eps;
  a.part = (float *)workspace;
  a.stats = stats ? stats : a.part + part_floats(a);
  hold(a, dtype, sb::kHeldThreads, sb::kHeldVectors);
  const hipError_t e = sb_launch_channels_norm(a, dtype, weight_dtype, (hipStream_t)stream);
  if (e != hipSuccess) return failf(SB_ELAUNCH, "group norm launch failed: %s", hipGetErrorString(e));
  return SB_OK;
}

extern "C" int group_norm_backward(const void *dy, const int64_t dy_stride[2], const void *x,
                                   const int64_t x_stride[2], const int64_t shape[3], int64_t groups,
                                   const float *stats, const void *gamma, const void *beta, int activation, int dtype,
                                   int weight_dtype, void *dx, const int64_t dx_stride[2], void *dgamma, void *dbeta,
                                   void *workspace, size_t workspace_bytes_, void *stream) {
  sb::ChanArgs a;
  int rc;
  const void *weights[4] = {gamma, beta, dgamma, dbeta};
  if ((rc = read_shape(shape, groups, dtype, a)) || (rc = check_types(activation, dtype, weight_dtype, weights, 4)) ||
      (rc = check_weights_apart(weights, weight_dtype, a.C)))
    return rc;
  if (a.N == 0 || a.S == 0) {
    a.N = a.S = a.chunks = 0; // the weights' gradients are zeros
    if (!dgamma && !dbeta) return SB_OK;
  } else {
    if (!stats || !sb::aligned(stats, 4)) return failf(SB_EARG, "stats must be device memory aligned to its element size");
    sb::Strided sx, sdy, so;
    if ((rc = read_positions("dy", dy, dy_stride, a, dtype, a.sdy, sdy)) ||
        (rc = read_positions("x", x, x_stride, a, dtype, a.sx, sx)) ||
        (rc = read_positions("dx", dx, dx_stride, a, dtype, a.sout, so)) ||
        (rc = check_output("dx", dx, so, "x", x, sx, dtype)) || (rc = check_output("dx", dx, so, "dy", dy, sdy, dtype)) ||
        (rc = check_workspace(workspace, workspace_bytes_, workspace_bytes(a))))
      return rc;
  }
  a.x = x;
  a.dy = dy;
  a.out = dx;
  a.gamma = gamma;
  a.beta = beta;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.silu = activation == SB_ACT_SILU;
  a.stats = const_cast<float *>(stats); // only read
  a.part = (float *)workspace;
  a.coef = a.part + part_floats(a);
  a.apply_chunk = a.chunk;
  a.apply_chunks = a.chunks;
  if (a.N) hold(a, dtype, sb::kHeldBackThreads, sb::kHeldBackVectors);
  const hipError_t e = sb_launch_channels_norm_backward(a, dtype, weight_dtype, (hipStream_t)stream);
  if (e != hipSuccess) return failf(SB_ELAUNCH, "group norm launch failed: %s", hipGetErrorString(e));
  return SB_OK;
}
