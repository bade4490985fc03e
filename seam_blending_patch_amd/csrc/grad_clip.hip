// grad_clip.hip -- the norm of a list of gradients, and clipping by it, gfx950.
//
// norm = sqrt(sum over all tensors of g^2), c = min(1, max_norm / (norm + eps)),
// out = g c.  Two passes: sums of squares of every chunk of every tensor, then
// each block adds all of those up, in the same order everywhere, and scales
// its chunk.  No atomics, so the same inputs give the same bits.
//
// Squares are formed and summed in 64 bits: they neither overflow nor vanish
// for any 32-bit gradient.  The factor is rounded to fp32 before it scales,
// unless it is below fp32's normal numbers, which would cost it bits.

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

// The tensor whose chunks hold chunk b: the last whose first chunk is at most
// b.  Every lane compares two of the table's entries, so that the search takes
// one memory latency (a binary search takes seven).
__device__ __forceinline__ int find_tensor(const ClipArgs &A, uint32_t b) {
  static_assert(kClipTensors == 128, "two entries a lane");
  const int lane = threadIdx.x & 63;
  const bool low = lane < A.tensors && A.begin[lane] <= b;
  const bool high = lane + 64 < A.tensors && A.begin[lane + 64] <= b;
  return __popcll(__ballot(low)) + __popcll(__ballot(high)) - 1;
}

// f(element, number of them, vector) for every vector of elements [e0, e1), kClipBatch
// of a thread's requested before the first is used
constexpr int kClipBatch = 4;
template <int DT, class F>
__device__ __forceinline__ void each_vector(const void *p, int64_t e0, int64_t e1, F f) {
  constexpr int V = kVec<DT>, STEP = kClipThreads * V;
  int64_t e = e0 + threadIdx.x * V;
  for (; e + (kClipBatch - 1) * STEP + V <= e1; e += kClipBatch * STEP) {
    Vec<16> v[kClipBatch];
#pragma unroll
    for (int i = 0; i < kClipBatch; ++i) v[i] = load_part<DT>(p, e + i * STEP, V);
#pragma unroll
    for (int i = 0; i < kClipBatch; ++i) f(e + i * STEP, V, v[i]);
  }
  for (; e < e1; e += STEP) {
    const int n = (int)min(e1 - e, (int64_t)V);
    f(e, n, load_part<DT>(p, e, n));
  }
}

template <int DT> __device__ __forceinline__ double chunk_squares(const void *p, int64_t e0, int64_t e1) {
  double s = 0.0;
  each_vector<DT>(p, e0, e1, [&](int64_t, int, const Vec<16> &v) {
    float f[kVec<DT>];
    unpack<DT, 16>(v, f);
#pragma unroll
    for (int k = 0; k < kVec<DT>; ++k) s = fma((double)f[k], (double)f[k], s);
  });
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

template <int DT, bool NT>
__device__ __forceinline__ void chunk_scale(const void *in, void *out, int64_t e0, int64_t e1, float c) {
  constexpr int V = kVec<DT>;
  each_vector<DT>(in, e0, e1, [&](int64_t e, int n, const Vec<16> &v) {
    float f[V];
    unpack<DT, 16>(v, f);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] *= c;
    store_part<DT, NT>(out, e, n, pack<DT, 16>(f));
  });
}

// 16-bit gradients into fp32 ones, 4 elements a thread: a wave's stores are one
// run of 1 KiB.  (With 8 elements a thread, in two stores 32 bytes apart from
// lane to lane, 251 M bf16 elements took 428 us past the caches; these 299.)
template <int DT, bool NT>
__device__ __forceinline__ void chunk_widen(const void *in, void *out, int64_t e0, int64_t e1, float c) {
  constexpr int STEP = kClipThreads * 4, BATCH = 2 * kClipBatch;
  const uint16_t *p = (const uint16_t *)in;
  auto scale = [&](int64_t e, int n, uint32_t w0, uint32_t w1) {
    Vec<16> v;
    const uint32_t b[4] = {w0 & 0xFFFFu, w0 >> 16, w1 & 0xFFFFu, w1 >> 16};
#pragma unroll
    for (int k = 0; k < 4; ++k) v.w[k] = __float_as_uint(widen<DT>(b[k]) * c);
    store_part<DT_F32, NT>(out, e, n, v);
  };
  int64_t e = e0 + threadIdx.x * 4;
  for (; e + (BATCH - 1) * STEP + 4 <= e1; e += BATCH * STEP) {
    u32x2_el2 w[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) w[i] = *reinterpret_cast<const u32x2_el2 *>(p + e + i * STEP);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) scale(e + i * STEP, 4, w[i].x, w[i].y);
  }
  for (; e < e1; e += STEP) {
    const int n = (int)min(e1 - e, (int64_t)4);
    uint32_t b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) b[k] = k < n ? p[e + k] : 0;
    scale(e, n, b[0] | b[1] << 16, b[2] | b[3] << 16);
  }
}

template <bool NT>
__device__ __forceinline__ void chunk_of(int types, const void *in, void *out, int64_t e0, int64_t e1, float c) {
  switch (types) {
  case DT_F32 | DT_F32 << 2: chunk_scale<DT_F32, NT>(in, out, e0, e1, c); break;
  case DT_F16 | DT_F16 << 2: chunk_scale<DT_F16, NT>(in, out, e0, e1, c); break;
  case DT_F16 | DT_F32 << 2: chunk_widen<DT_F16, NT>(in, out, e0, e1, c); break;
  case DT_BF16 | DT_F32 << 2: chunk_widen<DT_BF16, NT>(in, out, e0, e1, c); break;
  default: chunk_scale<DT_BF16, NT>(in, out, e0, e1, c); break;
  }
}

// A chunk scaled in 64 bits, an element a thread at a time: for factors that
// fp32 holds with fewer bits or not at all (norms 2^126 times the bound), while
// the products may be ordinary numbers.
template <int DT, int ODT>
__device__ __forceinline__ void chunk_scale_f64(const void *in, void *out, int64_t e0, int64_t e1, double by) {
  for (int64_t e = e0 + threadIdx.x; e < e1; e += kClipThreads) {
    const float f = widen<DT>(((const typename El<DT>::bits *)in)[e]);
    ((typename El<ODT>::bits *)out)[e] = (typename El<ODT>::bits)narrow<ODT>((float)(f * by));
  }
}

__device__ __forceinline__ void chunk_of_f64(int types, const void *in, void *out, int64_t e0, int64_t e1, double by) {
  switch (types) {
  case DT_F32 | DT_F32 << 2: chunk_scale_f64<DT_F32, DT_F32>(in, out, e0, e1, by); break;
  case DT_F16 | DT_F16 << 2: chunk_scale_f64<DT_F16, DT_F16>(in, out, e0, e1, by); break;
  case DT_F16 | DT_F32 << 2: chunk_scale_f64<DT_F16, DT_F32>(in, out, e0, e1, by); break;
  case DT_BF16 | DT_F32 << 2: chunk_scale_f64<DT_BF16, DT_F32>(in, out, e0, e1, by); break;
  default: chunk_scale_f64<DT_BF16, DT_BF16>(in, out, e0, e1, by); break;
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
  if (by > 0.0 && by < 0x1p-126) chunk_of_f64(A.types[t], A.in[t], A.out[t], e0, e1, by);
  else if (A.nt) chunk_of<true>(A.types[t], A.in[t], A.out[t], e0, e1, c);
  else chunk_of<false>(A.types[t], A.in[t], A.out[t], e0, e1, c);
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
