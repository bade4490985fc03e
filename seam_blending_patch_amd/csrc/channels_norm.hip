// channels_norm.hip -- group norm of channels-last activations with SiLU, and its
// gradient, for gfx950.
//
// A thread keeps one vector of channels and goes along the positions: whatever the
// group's channels, a block reads whole runs of a position's channels, and sums
// stay in registers by channel until the block's end.  Bound by memory.
#include <type_traits>

#include "sb_channels.h"
#include "sb_row.h"

namespace sb {
namespace {

// A block's columns and positions, and a thread's.
struct Place {
  int n, chunk, r, col; // sample, chunk of its positions; of a thread: its position in a turn and vector column
  int s0, s1;           // the chunk's positions
  bool on;              // (the threads that are left over when a turn's positions do not fill the block are off)
};
__device__ __forceinline__ Place place_of(const ChanArgs &a) {
  const uint32_t b = a.block0 + blockIdx.x, t = fdiv(b, a.div_slabs), slab = b - t * a.div_slabs.d;
  Place p;
  p.n = (int)fdiv(t, a.div_chunks);
  p.chunk = (int)(t - (uint32_t)p.n * a.div_chunks.d);
  p.s0 = p.chunk * a.chunk;
  p.s1 = min(p.s0 + a.chunk, a.S);
  p.r = (int)fdiv(threadIdx.x, a.div_CV);
  p.col = (int)threadIdx.x - p.r * a.CV + (int)slab * a.CV;
  p.on = p.r < a.RB && p.col < a.NV;
  return p;
}

// positions of a chunk of `len` that the thread with position r of a turn has
__device__ __forceinline__ int turns_of(int len, int r, int RB) { return len > r ? (len - r + RB - 1) / RB : 0; }

template <int DT> __device__ __forceinline__ float value_at(const void *p, int64_t e) {
  return widen<DT>(((const typename El<DT>::bits *)p)[e]);
}

// the first part of a group's mean: its first value.  Sums are taken of what is
// left, so a mean that is large against the spread costs no accuracy.
template <int DT> __device__ __forceinline__ float group_shift(const ChanArgs &a, int n, int g) {
  return value_at<DT>(a.x, n * a.sx.n + (int64_t)g * a.Cg);
}

// Statistics of a block's chunk by channel: batches of a thread's positions,
// each by two passes over its registers, merged (Chan, Golub & LeVeque); then the
// block's threads by a tree.
template <int DT, Cover C>
__global__ __launch_bounds__(kChanThreads) void stats_kernel(const ChanArgs a) {
  constexpr int V = kVec<DT>, R = kChanBatch;
  __shared__ float lds[2][kChanThreads * V];
  const Place p = place_of(a);
  const int e = p.col * V, len = p.s1 - p.s0;
  float K[V], mean[V], m2[V];
  int count = 0;
#pragma unroll
  for (int k = 0; k < V; ++k) mean[k] = m2[k] = 0.0f;
  if (p.on) {
#pragma unroll
    for (int k = 0; k < V; ++k)
      K[k] = group_shift<DT>(a, p.n, (int)fdiv((uint32_t)min(e + k, a.C - 1), a.div_Cg));
    const int turns = turns_of(len, p.r, a.RB);
    int64_t at = p.n * a.sx.n + (int64_t)(p.s0 + p.r) * a.sx.s;
    const int64_t step = a.RB * a.sx.s;
    const auto batch = [&](auto full, int m) {
      Vec<16> v[R];
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (decltype(full)::value || j < m) v[j] = request_row<DT, C>(a.x, at + j * step, e, a.C);
      float s[V];
#pragma unroll
      for (int k = 0; k < V; ++k) s[k] = 0.0f;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (decltype(full)::value || j < m) {
          settle_row<DT, C>(v[j], e, a.C);
          float f[V];
          unpack<DT, 16>(v[j], f);
#pragma unroll
          for (int k = 0; k < V; ++k) s[k] += f[k] - K[k];
        }
      const float rm = 1.0f / (float)m;
      float q[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        s[k] *= rm;
        q[k] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (decltype(full)::value || j < m) {
          float f[V];
          unpack<DT, 16>(v[j], f);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const float d = (f[k] - K[k]) - s[k];
            q[k] = __builtin_fmaf(d, d, q[k]);
          }
        }
      const float w = (float)m / (float)(count + m), wc = w * (float)count;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float d = s[k] - mean[k];
        mean[k] = __builtin_fmaf(d, w, mean[k]);
        m2[k] += __builtin_fmaf(d * d, wc, q[k]);
      }
      count += m;
      at += R * step;
    };
    int t = 0;
    for (; t + R <= turns; t += R) batch(std::true_type{}, R);
    if (t < turns) batch(std::false_type{}, turns - t);
  }
  // the threads of a column: the upper half of what is left hands over
  int top = 1;
  while (top < a.RB) top *= 2;
  for (int s = top / 2; s; s /= 2) {
    __syncthreads();
    if (p.on && p.r >= s && p.r < 2 * s) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        lds[0][k * kChanThreads + threadIdx.x] = mean[k];
        lds[1][k * kChanThreads + threadIdx.x] = m2[k];
      }
    }
    __syncthreads();
    if (p.on && p.r < s && p.r + s < a.RB) {
      // (all of the positions that r + s has merged, r + s + 2 s, ... among them)
      int theirs = 0;
      for (int r = p.r + s; r < a.RB; r += 2 * s) theirs += turns_of(len, r, a.RB);
      if (theirs) {
        const float w = (float)theirs / (float)(count + theirs), wc = w * (float)count;
        const int from = threadIdx.x + s * a.CV;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float d = lds[0][k * kChanThreads + from] - mean[k];
          mean[k] = __builtin_fmaf(d, w, mean[k]);
          m2[k] += __builtin_fmaf(d * d, wc, lds[1][k * kChanThreads + from]);
        }
        count += theirs;
      }
    }
  }
  if (p.on && p.r == 0) {
    float *to = a.part + ((int64_t)p.n * a.chunks + p.chunk) * 2 * a.C + e;
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (C != CUT || e + k < a.C) {
        to[k] = mean[k];
        to[a.C + k] = m2[k];
      }
  }
}

// a block's sum of one double each, in every thread
__device__ __forceinline__ double block_sum(double v, double *lds) {
#pragma unroll
  for (int k = 32; k; k >>= 1) v += __shfl_xor(v, k);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kChanThreads / 64; ++w) s += lds[w];
  return s;
}

// A group's chunks and channels merged: a block to a group.  64 bits: the sums
// are short and cost nothing.
template <int DT> __global__ __launch_bounds__(kChanThreads) void merge_kernel(const ChanArgs a) {
  __shared__ double lds[kChanThreads / 64];
  const int n = blockIdx.x / a.G, g = blockIdx.x - n * a.G, items = a.chunks * a.Cg;
  const float *part = a.part + (int64_t)n * a.chunks * 2 * a.C + g * a.Cg;
  const double total = (double)a.S * a.Cg;
  const auto count_of = [&](int chunk) { return (double)(min(a.S, (chunk + 1) * a.chunk) - chunk * a.chunk); };
  double s = 0.0;
  for (int i = threadIdx.x; i < items; i += kChanThreads) {
    const int chunk = (int)fdiv((uint32_t)i, a.div_Cg), c = i - chunk * a.Cg;
    s += count_of(chunk) * (double)part[(int64_t)chunk * 2 * a.C + c];
  }
  const double mean = block_sum(s, lds) / total;
  s = 0.0;
  for (int i = threadIdx.x; i < items; i += kChanThreads) {
    const int chunk = (int)fdiv((uint32_t)i, a.div_Cg), c = i - chunk * a.Cg;
    const double d = (double)part[(int64_t)chunk * 2 * a.C + c] - mean;
    s += (double)part[((int64_t)chunk * 2 + 1) * a.C + c] + count_of(chunk) * d * d;
  }
  const double var = block_sum(s, lds) / total;
  if (threadIdx.x == 0) {
    float *to = a.stats + ((int64_t)n * a.G + g) * 3;
    to[0] = group_shift<DT>(a, n, g);
    to[1] = (float)mean;
    to[2] = (float)(1.0 / sqrt(var + (double)a.eps));
  }
}

// 1 / (1 + exp(-z))
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

// What a thread keeps of its channels: h = ((x - K) - m) r, z = h gamma + beta.
template <int DT, int WT, Cover C> struct Channels {
  static constexpr int V = kVec<DT>;
  float K[V], m[V], r[V], gamma[V], beta[V];
  __device__ __forceinline__ void load(const ChanArgs &a, int n, int e) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = min(e + k, a.C - 1);
      const float *st = a.stats + ((int64_t)n * a.G + fdiv((uint32_t)c, a.div_Cg)) * 3;
      K[k] = st[0];
      m[k] = st[1];
      r[k] = st[2];
      gamma[k] = a.gamma ? value_at<WT>(a.gamma, c) : 1.0f;
      beta[k] = a.beta ? value_at<WT>(a.beta, c) : 0.0f;
    }
  }
  __device__ __forceinline__ float h(float x, int k) const { return ((x - K[k]) - m[k]) * r[k]; }
};

template <int DT, int WT, Cover C, bool SILU>
__global__ __launch_bounds__(kChanThreads) void apply_kernel(const ChanArgs a) {
  constexpr int V = kVec<DT>, R = kChanBatch;
  const Place p = place_of(a);
  if (!p.on) return;
  const int e = p.col * V;
  Channels<DT, WT, C> ch;
  ch.load(a, p.n, e);
  const int turns = turns_of(p.s1 - p.s0, p.r, a.RB);
  int64_t in = p.n * a.sx.n + (int64_t)(p.s0 + p.r) * a.sx.s, to = p.n * a.sout.n + (int64_t)(p.s0 + p.r) * a.sout.s;
  const int64_t si = a.RB * a.sx.s, so = a.RB * a.sout.s;
  for (int t = 0; t < turns; t += R, in += R * si, to += R * so) {
    Vec<16> v[R];
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (t + j < turns) v[j] = request_row<DT, C>(a.x, in + j * si, e, a.C);
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (t + j < turns) {
        settle_row<DT, C>(v[j], e, a.C);
        float f[V];
        unpack<DT, 16>(v[j], f);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float z = __builtin_fmaf(ch.h(f[k], k), ch.gamma[k], ch.beta[k]);
          f[k] = SILU ? z * logistic(z) : z;
        }
        store_row<DT, C>(a.out, to + j * so, e, a.C, pack<DT, 16>(f));
      }
  }
}

// g = dy act'(z), h: of one vector
template <int DT, int WT, Cover C, bool SILU>
__device__ __forceinline__ void gradient_of(const Channels<DT, WT, C> &ch, const Vec<16> &x, const Vec<16> &dy,
                                            float *g, float *h) {
  constexpr int V = kVec<DT>;
  unpack<DT, 16>(x, h);
  unpack<DT, 16>(dy, g);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    h[k] = ch.h(h[k], k);
    if constexpr (SILU) {
      const float z = __builtin_fmaf(h[k], ch.gamma[k], ch.beta[k]), s = logistic(z);
      g[k] *= s * __builtin_fmaf(z, 1.0f - s, 1.0f);
    }
  }
}

// Sums of g and g h by channel over a block's chunk.
template <int DT, int WT, Cover C, bool SILU>
__global__ __launch_bounds__(kChanThreads) void sums_kernel(const ChanArgs a) {
  constexpr int V = kVec<DT>, R = kChanBatch / 2;
  __shared__ float lds[2][kChanThreads * V];
  const Place p = place_of(a);
  const int e = p.col * V;
  float sg[V], sh[V];
#pragma unroll
  for (int k = 0; k < V; ++k) sg[k] = sh[k] = 0.0f;
  if (p.on) {
    Channels<DT, WT, C> ch;
    ch.load(a, p.n, e);
    const int turns = turns_of(p.s1 - p.s0, p.r, a.RB);
    int64_t ix = p.n * a.sx.n + (int64_t)(p.s0 + p.r) * a.sx.s, iy = p.n * a.sdy.n + (int64_t)(p.s0 + p.r) * a.sdy.s;
    const int64_t stx = a.RB * a.sx.s, sty = a.RB * a.sdy.s;
    for (int t = 0; t < turns; t += R, ix += R * stx, iy += R * sty) {
      Vec<16> v[R], w[R];
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (t + j < turns) {
          v[j] = request_row<DT, C>(a.x, ix + j * stx, e, a.C);
          w[j] = request_row<DT, C>(a.dy, iy + j * sty, e, a.C);
        }
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (t + j < turns) {
          settle_row<DT, C>(v[j], e, a.C);
          settle_row<DT, C>(w[j], e, a.C);
          float g[V], h[V];
          gradient_of<DT, WT, C, SILU>(ch, v[j], w[j], g, h);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            sg[k] += g[k];
            sh[k] = __builtin_fmaf(g[k], h[k], sh[k]);
          }
        }
    }
  }
  int top = 1;
  while (top < a.RB) top *= 2;
  for (int s = top / 2; s; s /= 2) {
    __syncthreads();
    if (p.on && p.r >= s && p.r < 2 * s) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        lds[0][k * kChanThreads + threadIdx.x] = sg[k];
        lds[1][k * kChanThreads + threadIdx.x] = sh[k];
      }
    }
    __syncthreads();
    if (p.on && p.r < s && p.r + s < a.RB) {
      const int from = threadIdx.x + s * a.CV;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        sg[k] += lds[0][k * kChanThreads + from];
        sh[k] += lds[1][k * kChanThreads + from];
      }
    }
  }
  if (p.on && p.r == 0) {
    float *to = a.part + ((int64_t)p.n * a.chunks + p.chunk) * 2 * a.C + e;
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (C != CUT || e + k < a.C) {
        to[k] = sg[k];
        to[a.C + k] = sh[k];
      }
  }
}

// The sums over a group (first N G blocks: means of gamma g and gamma g h), and
// over the samples by channel (a wave to a channel: dbeta and dgamma).
template <int WT> __global__ __launch_bounds__(kChanThreads) void gather_kernel(const ChanArgs a) {
  __shared__ double lds[kChanThreads / 64];
  if ((int)blockIdx.x < a.N * a.G) {
    const int n = blockIdx.x / a.G, g = blockIdx.x - n * a.G, items = a.chunks * a.Cg;
    const float *part = a.part + (int64_t)n * a.chunks * 2 * a.C + g * a.Cg;
    double s = 0.0, t = 0.0;
    for (int i = threadIdx.x; i < items; i += kChanThreads) {
      const int chunk = (int)fdiv((uint32_t)i, a.div_Cg), c = i - chunk * a.Cg;
      const double gamma = a.gamma ? (double)value_at<WT>(a.gamma, g * a.Cg + c) : 1.0;
      s += gamma * (double)part[(int64_t)chunk * 2 * a.C + c];
      t += gamma * (double)part[((int64_t)chunk * 2 + 1) * a.C + c];
    }
    s = block_sum(s, lds);
    t = block_sum(t, lds);
    if (threadIdx.x == 0) {
      const double total = (double)a.S * a.Cg;
      a.coef[blockIdx.x * 2] = (float)(s / total);
      a.coef[blockIdx.x * 2 + 1] = (float)(t / total);
    }
    return;
  }
  const int c = ((int)blockIdx.x - a.N * a.G) * (kChanThreads / 64) + (threadIdx.x >> 6);
  if (c >= a.C) return;
  double s = 0.0, t = 0.0;
  for (int i = threadIdx.x & 63; i < a.N * a.chunks; i += 64) {
    s += (double)a.part[(int64_t)i * 2 * a.C + c];
    t += (double)a.part[((int64_t)i * 2 + 1) * a.C + c];
  }
#pragma unroll
  for (int k = 32; k; k >>= 1) {
    s += __shfl_xor(s, k);
    t += __shfl_xor(t, k);
  }
  if ((threadIdx.x & 63) == 0) {
    typedef typename El<WT>::bits bits;
    if (a.dbeta) ((bits *)a.dbeta)[c] = (bits)narrow<WT>((float)s);
    if (a.dgamma) ((bits *)a.dgamma)[c] = (bits)narrow<WT>((float)t);
  }
}

// dx = r (gamma g - mean(gamma g) - h mean(gamma g h))
template <int DT, int WT, Cover C, bool SILU>
__global__ __launch_bounds__(kChanThreads) void gradient_kernel(const ChanArgs a) {
  constexpr int V = kVec<DT>, R = kChanBatch / 2;
  const Place p = place_of(a);
  if (!p.on) return;
  const int e = p.col * V;
  Channels<DT, WT, C> ch;
  ch.load(a, p.n, e);
  float mg[V], mh[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const float *co = a.coef + ((int64_t)p.n * a.G + fdiv((uint32_t)min(e + k, a.C - 1), a.div_Cg)) * 2;
    mg[k] = co[0];
    mh[k] = co[1];
  }
  const int turns = turns_of(p.s1 - p.s0, p.r, a.RB);
  int64_t ix = p.n * a.sx.n + (int64_t)(p.s0 + p.r) * a.sx.s, iy = p.n * a.sdy.n + (int64_t)(p.s0 + p.r) * a.sdy.s,
          to = p.n * a.sout.n + (int64_t)(p.s0 + p.r) * a.sout.s;
  const int64_t stx = a.RB * a.sx.s, sty = a.RB * a.sdy.s, so = a.RB * a.sout.s;
  for (int t = 0; t < turns; t += R, ix += R * stx, iy += R * sty, to += R * so) {
    Vec<16> v[R], w[R];
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (t + j < turns) {
        v[j] = request_row<DT, C>(a.x, ix + j * stx, e, a.C);
        w[j] = request_row<DT, C>(a.dy, iy + j * sty, e, a.C);
      }
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (t + j < turns) {
        settle_row<DT, C>(v[j], e, a.C);
        settle_row<DT, C>(w[j], e, a.C);
        float g[V], h[V];
        gradient_of<DT, WT, C, SILU>(ch, v[j], w[j], g, h);
#pragma unroll
        for (int k = 0; k < V; ++k)
          g[k] = ch.r[k] * (__builtin_fmaf(g[k], ch.gamma[k], -mg[k]) - h[k] * mh[k]);
        store_row<DT, C>(a.out, to + j * so, e, a.C, pack<DT, 16>(g));
      }
  }
}

// launches of as many blocks as a grid takes
template <class F> void over_blocks(ChanArgs a, F launch) {
  const int64_t blocks = (int64_t)a.N * a.chunks * a.slabs;
  for (int64_t b = 0; b < blocks; b += kMaxBlocksX) {
    a.block0 = (uint32_t)b;
    launch(a, dim3((unsigned)(blocks - b < kMaxBlocksX ? blocks - b : kMaxBlocksX)));
  }
}

template <int DT, int WT, Cover C, bool SILU> hipError_t forward(const ChanArgs &a, hipStream_t st) {
  const dim3 block(kChanThreads);
  over_blocks(a, [&](const ChanArgs &b, dim3 grid) { hipLaunchKernelGGL((stats_kernel<DT, C>), grid, block, 0, st, b); });
  hipLaunchKernelGGL((merge_kernel<DT>), dim3((unsigned)(a.N * a.G)), block, 0, st, a);
  over_blocks(a, [&](const ChanArgs &b, dim3 grid) {
    hipLaunchKernelGGL((apply_kernel<DT, WT, C, SILU>), grid, block, 0, st, b);
  });
  return hipGetLastError();
}

template <int DT, int WT, Cover C, bool SILU> hipError_t backward(const ChanArgs &a, hipStream_t st) {
  const dim3 block(kChanThreads);
  const unsigned waves = kChanThreads / 64, columns = a.dgamma || a.dbeta ? (a.C + waves - 1) / waves : 0;
  over_blocks(a, [&](const ChanArgs &b, dim3 grid) {
    hipLaunchKernelGGL((sums_kernel<DT, WT, C, SILU>), grid, block, 0, st, b);
  });
  if (a.N * a.G + columns)
    hipLaunchKernelGGL((gather_kernel<WT>), dim3((unsigned)(a.N * a.G) + columns), block, 0, st, a);
  over_blocks(a, [&](const ChanArgs &b, dim3 grid) {
    hipLaunchKernelGGL((gradient_kernel<DT, WT, C, SILU>), grid, block, 0, st, b);
  });
  return hipGetLastError();
}

template <bool BACK, int DT, int WT, Cover C> hipError_t launch(const ChanArgs &a, hipStream_t st) {
  if constexpr (BACK) return a.silu ? backward<DT, WT, C, true>(a, st) : backward<DT, WT, C, false>(a, st);
  else return a.silu ? forward<DT, WT, C, true>(a, st) : forward<DT, WT, C, false>(a, st);
}
template <bool BACK, int DT> hipError_t launch(const ChanArgs &a, int wdtype, hipStream_t st) {
  const bool cut = a.C % kVec<DT> != 0;
  if (wdtype == DT_F32) return cut ? launch<BACK, DT, DT_F32, CUT>(a, st) : launch<BACK, DT, DT_F32, WHOLE>(a, st);
  return cut ? launch<BACK, DT, DT, CUT>(a, st) : launch<BACK, DT, DT, WHOLE>(a, st);
}
template <bool BACK> hipError_t launch(const ChanArgs &a, int dtype, int wdtype, hipStream_t st) {
  if (dtype == DT_F32) return launch<BACK, DT_F32>(a, wdtype, st);
  if (dtype == DT_F16) return launch<BACK, DT_F16>(a, wdtype, st);
  return launch<BACK, DT_BF16>(a, wdtype, st);
}

} // namespace
} // namespace sb

hipError_t sb_launch_channels_norm(const sb::ChanArgs &a, int dtype, int wdtype, hipStream_t st) {
  return sb::launch<false>(a, dtype, wdtype, st);
}
hipError_t sb_launch_channels_norm_backward(const sb::ChanArgs &a, int dtype, int wdtype, hipStream_t st) {
  return sb::launch<true>(a, dtype, wdtype, st);
}
