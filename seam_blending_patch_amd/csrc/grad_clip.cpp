// grad_clip.cpp -- host side of grad_norm and grad_norm_clip: argument checks,
// the split of the tensors into chunks, and launches of at most kClipTensors
// tensors whose table travels as a kernel argument (no copy to the device, so
// the calls can be captured in a graph).  No device memory is allocated and the
// stream is never synchronised.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>
#include <memory>
#include <new>

#include "sb_host.h"
#include "sb_transformer.h"

using sb::failf;

namespace {

constexpr int64_t kMaxTensors = 1 << 16; // every block adds up a sum of each
constexpr int64_t kMaxElements = (int64_t)1 << 44; // over all tensors

struct ClipPlan {
  int64_t chunk, chunks;
};

int plan_clip(const int64_t *numels, int64_t n, ClipPlan &p) {
  if (n < 0 || n > kMaxTensors) return failf(SB_EGEOM, "0..2^16 tensors (got %lld)", (long long)n);
  if (n > 0 && !numels) return failf(SB_EARG, "null element counts");
  int64_t total = 0;
  for (int64_t k = 0; k < n; ++k) {
    if (numels[k] < 0) return failf(SB_EARG, "tensor %lld: negative element count", (long long)k);
    if (numels[k] > kMaxElements - total) return failf(SB_EGEOM, "more than 2^44 elements");
    total += numels[k];
  }
  // Chunks of 8192 elements, longer where that would be more than 4096 of
  // them.  First pass and second, us: 4.7 M fp32 elements that stay at 4096 a
  // chunk 6.4 + 4.6, at 8192 6.2 + 3.7, at 16384 6.4 + 3.3, and 22.6 M fp32 ones
  // into others 23 + 36, 23 + 33 and 24 + 32; 251 M bf16 ones into fp32 at most
  // 2048, 4096 and 8192 chunks 90 + 312, 86 + 299 and 85 + 318, 47 M 17 + 46,
  // 18 + 51 and 17 + 56 (every block adds up all chunks' sums).
  constexpr int64_t step = sb::kClipThreads * 8;
  p.chunk = std::max<int64_t>(8192, (total / 4096 + step - 1) / step * step);
  p.chunks = 0;
  for (int64_t k = 0; k < n; ++k) p.chunks += (numels[k] + p.chunk - 1) / p.chunk;
  return SB_OK;
}

// A tensor's bytes, and its place in the list.
struct Run {
  uintptr_t begin, end;
  int64_t k;
};

// What is written shares no byte with anything else that the call reads or
// writes: blocks scale and read in any order.  (An output over its own gradient
// is the caller's check.)
int check_written(const void *const *grads, void *const *outs, const int64_t *numels, const int *dtypes,
                  const int *out_dtypes, int64_t n) {
  auto run = [&](int64_t k, bool out) {
    const uintptr_t p = out ? (uintptr_t)outs[k] : (uintptr_t)grads[k];
    return Run{p, p + (uintptr_t)(numels[k] * sb::elem_bytes(out ? out_dtypes[k] : dtypes[k])), k};
  };
  const std::unique_ptr<Run[]> held(new (std::nothrow) Run[n > 0 ? n : 1]);
  if (!held) return failf(SB_EGEOM, "no host memory for the table of %lld tensors", (long long)n);
  Run *const first = held.get(), *last = first;
  bool ascending = true; // views of a bucket mostly are
  for (int64_t k = 0; k < n; ++k) {
    if (numels[k] == 0) continue;
    *last = run(k, outs != nullptr);
    ascending = ascending && (last == first || last[-1].end <= last->begin);
    ++last;
  }
  if (!ascending) {
    std::sort(first, last, [](const Run &a, const Run &b) { return a.begin < b.begin; });
    for (const Run *r = first + 1; r < last; ++r)
      if (r->begin < r[-1].end) {
        const char *what = outs ? "output" : "gradient";
        return failf(SB_EARG, "%s %lld shares memory with %s %lld, and both are written", what, (long long)r->k, what,
                     (long long)r[-1].k);
      }
  }
  if (!outs) return SB_OK;
  for (int64_t k = 0; k < n; ++k) {
    if (numels[k] == 0) continue;
    const Run g = run(k, false);
    const Run *r = std::upper_bound(first, last, g.begin, [](uintptr_t p, const Run &a) { return p < a.end; });
    for (; r < last && r->begin < g.end; ++r)
      if (r->k != k)
        return failf(SB_EARG, "output %lld shares memory with gradient %lld", (long long)r->k, (long long)k);
  }
  return SB_OK;
}

int clip_call(const void *const *grads, void *const *outs, const int64_t *numels, const int *dtypes,
              const int *out_dtypes, int64_t n, bool scale, float max_norm, float eps, float *norm, void *workspace,
              size_t workspace_bytes, void *stream) {
  ClipPlan p;
  int rc = plan_clip(numels, n, p);
  if (rc) return rc;
  if (!norm || !sb::aligned(norm, 4)) return failf(SB_EARG, "norm must be a 4-byte aligned device pointer");
  if (scale && !(max_norm >= 0.0f)) return failf(SB_EARG, "max_norm must be >= 0");
  if (scale && (!(eps >= 0.0f) || eps == __builtin_inff())) return failf(SB_EARG, "eps must be finite and >= 0");
  if (n > 0 && (!grads || !dtypes || (outs && !out_dtypes))) return failf(SB_EARG, "null tensor table");
  for (int64_t k = 0; k < n; ++k) {
    if (!sb::known_dtype(dtypes[k])) return failf(SB_EARG, "tensor %lld: unknown dtype %d", (long long)k, dtypes[k]);
    if (outs && out_dtypes[k] != dtypes[k] && out_dtypes[k] != SB_F32)
      return failf(SB_EARG, "tensor %lld: the output must be of the gradient's dtype or fp32", (long long)k);
    if (numels[k] == 0) continue;
    if (!grads[k] || !sb::aligned(grads[k], sb::elem_bytes(dtypes[k])))
      return failf(SB_EARG, "gradient %lld is null or not aligned to its element size", (long long)k);
    if (!outs) continue;
    if (!outs[k] || !sb::aligned(outs[k], sb::elem_bytes(out_dtypes[k])))
      return failf(SB_EARG, "output %lld is null or not aligned to its element size", (long long)k);
    const uintptr_t g = (uintptr_t)grads[k], o = (uintptr_t)outs[k];
    const uintptr_t gn = (uintptr_t)(numels[k] * sb::elem_bytes(dtypes[k]));
    const uintptr_t on = (uintptr_t)(numels[k] * sb::elem_bytes(out_dtypes[k]));
    if (!(g == o && dtypes[k] == out_dtypes[k]) && g < o + on && o < g + gn)
      return failf(SB_EARG, "output %lld overlaps its gradient without being it", (long long)k);
  }
  if (scale && (rc = check_written(grads, outs, numels, dtypes, out_dtypes, n))) return rc;
  if (!workspace || !sb::aligned(workspace, 16)) return failf(SB_EARG, "workspace must be 16-byte aligned device memory");
  const size_t need = (size_t)std::max<int64_t>(p.chunks, 2) * sizeof(double);
  if (workspace_bytes < need)
    return failf(SB_EWORKSPACE, "workspace too small: %zu bytes given, %zu needed", workspace_bytes, need);

  // Outputs past the caches where gradients and outputs are more than the
  // last-level one holds: the gradients stay in it, and the next call's first
  // pass does not wait for the outputs to leave it.  Below that, an update that
  // reads the outputs next finds them there.  us with the hint and without, the
  // clip alone and (with such an update behind it): fp32 into fp32, 181 MB moved
  // 51 / 58 (105 / 102), 240 MB 67 / 79 (135 / 138), 300 MB 85 / 103 (165 / 180),
  // 1 GB 300 / 307 (576 / 585); bf16 into fp32, 181 MB 52 / 61 (121 / 115), 240 MB
  // 64 / 75 (153 / 165), 300 MB 77 / 101 (187 / 214), 1 GB 279 / 281 (638 / 643).
  int64_t moved = 0;
  for (int64_t k = 0; k < n; ++k)
    moved += numels[k] * (sb::elem_bytes(dtypes[k]) + (outs ? sb::elem_bytes(out_dtypes[k]) : 0));
  sb::ClipArgs a;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t done = 0, k = 0;
    bool first = true;
    while (k < n) {
      std::memset(&a, 0, sizeof a);
      a.chunk = p.chunk;
      a.max_norm = max_norm;
      a.eps = eps;
      a.nt = moved >= sb::kLastLevelBytes;
      uint32_t c = 0;
      while (k < n && a.tensors < sb::kClipTensors) {
        if (numels[k] > 0) {
          const int t = a.tensors++;
          a.in[t] = grads[k];
          a.out[t] = outs ? outs[k] : const_cast<void *>(grads[k]);
          a.n[t] = numels[k];
          a.begin[t] = c;
          a.types[t] = (uint8_t)(dtypes[k] | (outs ? out_dtypes[k] : dtypes[k]) << 2);
          c += (uint32_t)((numels[k] + p.chunk - 1) / p.chunk);
        }
        ++k;
      }
      if (a.tensors == 0) break;
      a.begin[a.tensors] = c;
      hipError_t e;
      if (pass == 0) {
        a.partials = (double *)workspace + done;
        e = sb_launch_square_sums(a, c, (hipStream_t)stream);
      } else {
        a.partials = (double *)workspace;
        a.npartials = (int32_t)p.chunks;
        a.norm = first ? norm : nullptr;
        e = sb_launch_clip(a, c, (hipStream_t)stream);
      }
      if (e != hipSuccess) return failf(SB_ELAUNCH, "gradient norm launch failed: %s", hipGetErrorString(e));
      done += c;
      first = false;
    }
    if (pass == 0 && (!scale || p.chunks == 0)) { // the norm alone
      std::memset(&a, 0, sizeof a);
      a.partials = (double *)workspace;
      a.npartials = (int32_t)p.chunks;
      a.norm = norm;
      const hipError_t e = sb_launch_clip(a, 1, (hipStream_t)stream);
      if (e != hipSuccess) return failf(SB_ELAUNCH, "gradient norm launch failed: %s", hipGetErrorString(e));
      break;
    }
  }
  return SB_OK;
}

} // namespace

extern "C" size_t grad_norm_workspace_bytes(const int64_t *numels, int64_t n) {
  ClipPlan p;
  if (plan_clip(numels, n, p)) return 0;
  return (size_t)std::max<int64_t>(p.chunks, 2) * sizeof(double);
}

extern "C" int grad_norm(const void *const *grads, const int64_t *numels, const int *dtypes, int64_t n, float *norm,
                         void *workspace, size_t workspace_bytes, void *stream) {
  return clip_call(grads, nullptr, numels, dtypes, nullptr, n, false, 0.0f, 0.0f, norm, workspace, workspace_bytes,
                   stream);
}

extern "C" int grad_norm_clip(const void *const *grads, void *const *outs, const int64_t *numels, const int *dtypes,
                              const int *out_dtypes, int64_t n, float max_norm, float eps, float *norm,
                              void *workspace, size_t workspace_bytes, void *stream) {
  return clip_call(grads, outs, numels, dtypes, out_dtypes, n, true, max_norm, eps, norm, workspace, workspace_bytes,
                   stream);
}
