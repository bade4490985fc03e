// grad_clip.hip -- the norm of a list of gradients, and clipping by it, gfx950.
//
// norm = sqrt(sum over all tensors of g^2), c = min(1, max_norm / (norm + eps)),
// out = g c.  Two passes: sums of squares of every chunk of every tensor, then
// each block adds all of those up, in the same order everywhere, and scales
// its chunk.  No atomics, so the same inputs give the same bits.
//
// Squares are formed and summed in 64 bits: they neither overflow nor vanish
// for any 32-bit gradient.

#include "sb_row.h"
#include "sb_transformer.h"

namespace sb {

__device__ __forceinline__ double block_sum_f64(double v) {
  __shared__ double lds[kClipThreads / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < kClipThreads / 64; ++w) v += lds[w];
  return v;
}

// the tensor whose chunks hold chunk b: the last whose first chunk is at most b
// (tensors without elements have no chunks: the next one starts at the same)
__device__ __forceinline__ int find_tensor(const ClipArgs &A, uint32_t b) {
  int lo = 0, hi = A.tensors; // begin[lo] <= b < begin[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (A.begin[mid] <= b) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int DT> __device__ __forceinline__ double chunk_squares(const void *p, int64_t e0, int64_t e1) {
  constexpr int V = kVec<DT>;
  double s = 0.0;
  for (int64_t e = e0 + threadIdx.x * V; e < e1; e += kClipThreads * V) {
    float f[V];
    load_floats<DT, V>(p, e, (int)min(e1 - e, (int64_t)V), f);
#pragma unroll
    for (int k = 0; k < V; ++k) s = fma((double)f[k], (double)f[k], s);
  }
  return s;
}

__global__ __launch_bounds__(kClipThreads) void square_sums_kernel(const ClipArgs A) {
  const int t = find_tensor(A, blockIdx.x);
  const int64_t e0 = (int64_t)(blockIdx.x - A.begin[t]) * A.chunk, e1 = min(e0 + A.chunk, A.n[t]);
  double s;
  switch (A.types[t] & 3) {
  case DT_F32: s = chunk_squares<DT_F32>(A.in[t], e0, e1); break;
  case DT_F16: s = chunk_squares<DT_F16>(A.in[t], e0, e1); break;
  default: s = chunk_squares<DT_BF16>(A.in[t], e0, e1); break;
  }
  s = block_sum_f64(s);
  if (threadIdx.x == 0) A.partials[blockIdx.x] = s;
}

template <int DT, int ODT>
__device__ __forceinline__ void chunk_scale(const void *in, void *out, int64_t e0, int64_t e1, float c) {
  constexpr int V = kVec<DT>, OV = kVec<ODT>;
  for (int64_t e = e0 + threadIdx.x * V; e < e1; e += kClipThreads * V) {
    const int n = (int)min(e1 - e, (int64_t)V);
    float f[V];
    load_floats<DT, V>(in, e, n, f);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] *= c;
#pragma unroll
    for (int k = 0; k < V; k += OV) store_part<ODT>(out, e + k, n - k, pack<ODT, 16>(f + k));
  }
}

__global__ __launch_bounds__(kClipThreads) void clip_kernel(const ClipArgs A) {
  double s = 0.0;
  for (int i = threadIdx.x; i < A.npartials; i += kClipThreads) s += A.partials[i];
  const double norm = sqrt(block_sum_f64(s));
  if (A.norm && blockIdx.x == 0 && threadIdx.x == 0) *A.norm = (float)norm;
  if (A.tensors == 0) return;
  const double by = (double)A.max_norm / (norm + (double)A.eps);
  const float c = by >= 1.0 ? 1.0f : (float)by; // a norm that is no number stays one
  const int t = find_tensor(A, blockIdx.x);
  if (c == 1.0f && A.in[t] == A.out[t]) return; // in place and nothing to scale
  const int64_t e0 = (int64_t)(blockIdx.x - A.begin[t]) * A.chunk, e1 = min(e0 + A.chunk, A.n[t]);
  switch (A.types[t]) {
  case DT_F32 | DT_F32 << 2: chunk_scale<DT_F32, DT_F32>(A.in[t], A.out[t], e0, e1, c); break;
  case DT_F16 | DT_F16 << 2: chunk_scale<DT_F16, DT_F16>(A.in[t], A.out[t], e0, e1, c); break;
  case DT_F16 | DT_F32 << 2: chunk_scale<DT_F16, DT_F32>(A.in[t], A.out[t], e0, e1, c); break;
  case DT_BF16 | DT_F32 << 2: chunk_scale<DT_BF16, DT_F32>(A.in[t], A.out[t], e0, e1, c); break;
  default: chunk_scale<DT_BF16, DT_BF16>(A.in[t], A.out[t], e0, e1, c); break;
  }
}

} // namespace sb

hipError_t sb_launch_square_sums(const sb::ClipArgs &a, unsigned blocks, hipStream_t st) {
  hipLaunchKernelGGL(sb::square_sums_kernel, dim3(blocks), dim3(sb::kClipThreads), 0, st, a);
  return hipGetLastError();
}

hipError_t sb_launch_clip(const sb::ClipArgs &a, unsigned blocks, hipStream_t st) {
  hipLaunchKernelGGL(sb::clip_kernel, dim3(blocks), dim3(sb::kClipThreads), 0, st, a);
  return hipGetLastError();
}
