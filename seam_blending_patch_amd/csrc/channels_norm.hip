// channels_norm.hip -- group norm of channels-last activations with SiLU, and its
// gradient, for gfx950.
//
// A thread keeps one vector of channels and goes along the positions: whatever the
// group's channels, a block reads whole runs of a position's channels, and sums
// stay in registers by channel until the block's end.  Bound by memory: two samples
// of 512 x 512 x 256 fp16 145 us a call (kernels under the profiler: sums 53, merge 6, result
// 100 us: 5.1 and 5.4 TB/s).  The gradient of 256 x 256 x 512 bf16 81 us (37, 7 and 39 us,
// 3.6 and 5.2 TB/s: two blocks to a CU do not hide the sums' vector work).  A second
// reading of x (and dy) is the price of groups that no block holds.
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
  const uint32_t at = a.block0 + blockIdx.x, b = a.last ? a.last - at : at, t = fdiv(b, a.div_slabs), slab = b - t * a.div_slabs.d;
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

// A mean as the unevaluated sum of two floats, so that one that is large against the
// spread costs no accuracy: moved on by d, and made up again so that the first is the
// mean in fp32.
__device__ __forceinline__ void move_mean(float &hi, float &lo, float d) {
  lo += d;
  const float s = hi + lo, back = s - hi;
  lo = (hi - (s - back)) + (lo - back); // (what the sum's rounding left out, whichever is larger)
  hi = s;
}

// Statistics of a block's chunk by channel: batches of a thread's positions,
// each by two passes over its registers about its first value, merged (Chan, Golub &
// LeVeque); then the block's threads by a tree.  A value far out costs digits of its
// own batch alone, 8 positions of a channel.
template <int DT, Cover C>
__global__ __launch_bounds__(kChanThreads) void stats_kernel(const ChanArgs a) {
  constexpr int V = kVec<DT>, R = kChanBatch;
  __shared__ float lds[3][kChanThreads * V];
  const Place p = place_of(a);
  const int e = p.col * V, len = p.s1 - p.s0;
  float hi[V], lo[V], m2[V];
  int count = 0;
#pragma unroll
  for (int k = 0; k < V; ++k) hi[k] = lo[k] = m2[k] = 0.0f;
  if (p.on) {
    const int turns = turns_of(len, p.r, a.RB);
    int64_t at = p.n * a.sx.n + (int64_t)(p.s0 + p.r) * a.sx.s;
    const int64_t step = a.RB * a.sx.s;
    const auto batch = [&](auto full, int m) {
      Vec<16> v[R];
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (decltype(full)::value || j < m) v[j] = request_row<DT, C>(a.x, at + j * step, e, a.C);
      float K[V], s[V];
#pragma unroll
      for (int k = 0; k < V; ++k) s[k] = 0.0f;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (decltype(full)::value || j < m) {
          settle_row<DT, C>(v[j], e, a.C);
          float f[V];
          unpack<DT, 16>(v[j], f);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            if (j == 0) K[k] = f[k];
            else s[k] += f[k] - K[k];
          }
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
      if (count == 0) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          hi[k] = K[k];
          move_mean(hi[k], lo[k], s[k]);
          m2[k] = q[k];
        }
      } else {
        const float w = (float)m / (float)(count + m), wc = w * (float)count;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float d = (K[k] - hi[k]) + (s[k] - lo[k]);
          move_mean(hi[k], lo[k], d * w);
          m2[k] += __builtin_fmaf(d * d, wc, q[k]);
        }
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
        lds[0][k * kChanThreads + threadIdx.x] = hi[k];
        lds[1][k * kChanThreads + threadIdx.x] = lo[k];
        lds[2][k * kChanThreads + threadIdx.x] = m2[k];
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
          const float d = (lds[0][k * kChanThreads + from] - hi[k]) + (lds[1][k * kChanThreads + from] - lo[k]);
          move_mean(hi[k], lo[k], d * w);
          m2[k] += __builtin_fmaf(d * d, wc, lds[2][k * kChanThreads + from]);
        }
        count += theirs;
      }
    }
  }
  if (p.on && p.r == 0) {
    float *to = a.part + ((int64_t)p.n * a.chunks + p.chunk) * 3 * a.C + e;
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (C != CUT || e + k < a.C) {
        to[k] = hi[k];
        to[a.C + k] = lo[k];
        to[2 * a.C + k] = m2[k];
      }
  }
}

// a block's sums of two doubles each, in every thread
__device__ __forceinline__ void block_sums(double &u, double &v, double (*lds)[2]) {
#pragma unroll
  for (int k = 32; k; k >>= 1) {
    u += __shfl_xor(u, k);
    v += __shfl_xor(v, k);
  }
  if ((threadIdx.x & 63) == 0) {
    lds[threadIdx.x >> 6][0] = u;
    lds[threadIdx.x >> 6][1] = v;
  }
  __syncthreads();
  u = v = 0.0;
  for (int w = 0; w < (int)blockDim.x / 64; ++w) {
    u += lds[w][0];
    v += lds[w][1];
  }
}

// Calls f(chunk, channel of the group, partials) with a group's partials (W of a chunk
// and channel), 8 of a thread on their way at a time.
template <int W, class F> __device__ __forceinline__ void over_partials(const ChanArgs &a, int n, int g, F f) {
  const float *part = a.part + (int64_t)n * a.chunks * W * a.C + g * a.Cg;
  const int items = a.chunks * a.Cg;
  for (int i0 = threadIdx.x; i0 < items; i0 += 8 * kMergeThreads) {
    float v[8][W];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = min(i0 + j * kMergeThreads, items - 1), chunk = (int)fdiv((uint32_t)i, a.div_Cg);
      const float *at = part + (int64_t)chunk * W * a.C + (i - chunk * a.Cg);
#pragma unroll
      for (int w = 0; w < W; ++w) v[j][w] = at[w * a.C];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * kMergeThreads;
      if (i < items) {
        const int chunk = (int)fdiv((uint32_t)i, a.div_Cg);
        f(chunk, i - chunk * a.Cg, v[j]);
      }
    }
  }
}

// A group's chunks and channels merged: a block to a group.  In 64 bits the merge of
// many sets may be taken by sums of squares, of what the group's first value leaves of
// the means: that is either near them or, far out of n values, a deviation of its
// distance over sqrt(n) by itself (n up to 2^30 leaves 2^-23 of the variance).
template <int DT> __global__ __launch_bounds__(kMergeThreads) void merge_kernel(const ChanArgs a) {
  __shared__ double lds[kMergeThreads / 64][2];
  const int n = blockIdx.x / a.G, g = blockIdx.x - n * a.G;
  const double total = (double)a.S * a.Cg;
  const double first = value_at<DT>(a.x, n * a.sx.n + (int64_t)g * a.Cg);
  double s = 0.0, t = 0.0;
  over_partials<3>(a, n, g, [&](int chunk, int, const float (&v)[3]) {
    const double count = min(a.S, (chunk + 1) * a.chunk) - chunk * a.chunk, m = ((double)v[0] - first) + (double)v[1];
    s += count * m;
    t += (double)v[2] + count * m * m;
  });
  block_sums(s, t, lds);
  if (threadIdx.x == 0) {
    const double rest = s / total, off = t / total - rest * rest, var = off < 0.0 ? 0.0 : off, mean = first + rest; // (NaN stays)
    float *to = a.stats + ((int64_t)n * a.G + g) * 3;
    to[0] = (float)mean;
    to[1] = (float)(mean - (double)to[0]);
    to[2] = (float)(1.0 / sqrt(var + (double)a.eps));
  }
}

// 1 / (1 + exp(-z))
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

// What a thread keeps of its channels: h = ((x - K) - m) r, z = h gamma + beta.
template <int DT, int WT> struct Channels {
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

template <int DT, int WT, Cover C, bool SILU, bool FAR>
__global__ __launch_bounds__(kChanThreads) void apply_kernel(const ChanArgs a) {
  constexpr int V = kVec<DT>, R = kChanBatch;
  const Place p = place_of(a);
  if (!p.on) return;
  const int e = p.col * V;
  Channels<DT, WT> ch;
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
        store_row<DT, C, FAR>(a.out, to + j * so, e, a.C, pack<DT, 16>(f));
      }
  }
}

// g = dy act'(z), h: of one vector
template <int DT, int WT, bool SILU>
__device__ __forceinline__ void gradient_of(const Channels<DT, WT> &ch, const Vec<16> &x, const Vec<16> &dy,
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
    Channels<DT, WT> ch;
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
          gradient_of<DT, WT, SILU>(ch, v[j], w[j], g, h);
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

// The sums over a group (first N G blocks: means of gamma g and gamma g h), and by
// channel over the samples (a block to 64 channels: dbeta and dgamma).
template <int WT> __global__ __launch_bounds__(kMergeThreads) void gather_kernel(const ChanArgs a) {
  constexpr int W = kMergeThreads / 64;
  __shared__ double lds[W][2];
  __shared__ double sums[W][2][64];
  if ((int)blockIdx.x < a.N * a.G) {
    const int n = blockIdx.x / a.G, g = blockIdx.x - n * a.G;
    double s = 0.0, t = 0.0;
    over_partials<2>(a, n, g, [&](int, int c, const float (&v)[2]) {
      const double gamma = a.gamma ? (double)value_at<WT>(a.gamma, g * a.Cg + c) : 1.0;
      s += gamma * (double)v[0];
      t += gamma * (double)v[1];
    });
    block_sums(s, t, lds);
    if (threadIdx.x == 0) {
      const double total = (double)a.S * a.Cg;
      a.coef[blockIdx.x * 2] = (float)(s / total);
      a.coef[blockIdx.x * 2 + 1] = (float)(t / total);
    }
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = ((int)blockIdx.x - a.N * a.G) * 64 + lane;
  const int rows = a.N * a.chunks;
  double s = 0.0, t = 0.0;
  if (c < a.C) {
    for (int i0 = wave; i0 < rows; i0 += 8 * W) {
      float u[8], v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float *at = a.part + (int64_t)min(i0 + j * W, rows - 1) * 2 * a.C + c;
        u[j] = at[0];
        v[j] = at[a.C];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + j * W < rows) {
          s += (double)u[j];
          t += (double)v[j];
        }
    }
  }
  sums[wave][0][lane] = s;
  sums[wave][1][lane] = t;
  __syncthreads();
  if (wave < 2 && c < a.C) { // the first wave dbeta, the second dgamma
    double sum = 0.0;
    for (int w = 0; w < W; ++w) sum += sums[w][wave][lane];
    typedef typename El<WT>::bits bits;
    void *to = wave ? a.dgamma : a.dbeta;
    if (to) ((bits *)to)[c] = (bits)narrow<WT>((float)sum);
  }
}

// dx = r (gamma g - mean(gamma g) - h mean(gamma g h))
template <int DT, int WT, Cover C, bool SILU, bool FAR>
__global__ __launch_bounds__(kChanThreads) void gradient_kernel(const ChanArgs a) {
  constexpr int V = kVec<DT>, R = kChanBatch / 2;
  const Place p = place_of(a);
  if (!p.on) return;
  const int e = p.col * V;
  Channels<DT, WT> ch;
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
        gradient_of<DT, WT, SILU>(ch, v[j], w[j], g, h);
#pragma unroll
        for (int k = 0; k < V; ++k)
          g[k] = ch.r[k] * (__builtin_fmaf(g[k], ch.gamma[k], -mg[k]) - h[k] * mh[k]);
        store_row<DT, C, FAR>(a.out, to + j * so, e, a.C, pack<DT, 16>(g));
      }
  }
}

// ---------------------------------------------------------------------------
// Groups that a block holds in registers: one launch, x read once.  64 samples of
// 1024 x 320 bf16 39 us against 53 in passes over blocks, 8 of 256 x 1280 fp16 10
// against 20 (the host's work of a call); 2 of 1024 x 320 fp16, where 16 blocks have
// 80 KiB each to fetch, 13.2 against 15.
// ---------------------------------------------------------------------------
// A block's channels c0 .. c0 + CS of sample n; a thread has vector column col of
// positions r, r + RB, ...
struct Held {
  int n, c0, r, col, RB;
  bool on;
  template <int THREADS> static __device__ __forceinline__ Held of(const ChanArgs &a) {
    const int per = a.G / a.sg, cv = (int)a.div_CVs.d;
    Held p;
    p.n = blockIdx.x / per;
    p.c0 = (blockIdx.x - p.n * per) * a.CS;
    p.RB = THREADS / cv;
    p.r = (int)fdiv(threadIdx.x, a.div_CVs);
    p.col = threadIdx.x - p.r * cv;
    p.on = p.r < p.RB;
    return p;
  }
};

// The values of K sums by channel of every thread, added up over the block for each
// of its groups (at most 8): within a wave without memory, then over the waves.
template <int K, int V, int THREADS>
__device__ __forceinline__ void group_sums(int sg, const int (&group)[V], const float (&v)[K][V], float (*lds)[8][THREADS / 64],
                                           float (*out)[8]) {
  constexpr int W = THREADS / 64;
  for (int g = 0; g < sg; ++g) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < V; ++k) s += group[k] == g ? v[j][k] : 0.0f;
      s = lanes_sum<64>(s);
      if ((threadIdx.x & 63) == 0) lds[j][g][threadIdx.x >> 6] = s;
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < sg * K) {
    const int j = threadIdx.x / sg, g = threadIdx.x - j * sg;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) s += lds[j][g][w];
    out[j][g] = s;
  }
  __syncthreads();
}

// N weights from channel e on
template <int WT, int N> __device__ __forceinline__ void weights_of(const void *p, int e, float fill, float (&f)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) f[k] = p ? value_at<WT>(p, e + k) : fill;
}

template <int DT, int WT, bool SILU> __global__ __launch_bounds__(kHeldThreads) void held_kernel(const ChanArgs a) {
  constexpr int V = kVec<DT>, NV = kHeldVectors;
  __shared__ float lds[2][8][kHeldThreads / 64], sums[3][2][8];
  const Held p = Held::of<kHeldThreads>(a);
  const int e = p.c0 + (p.on ? p.col * V : 0), row = p.on ? p.r : 0;
  Vec<16> v[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) // (positions past the end: the last one, left out below)
    v[j] = load_part<DT>(a.x, p.n * a.sx.n + (int64_t)min(row + j * p.RB, a.S - 1) * a.sx.s + e, V);
  float gamma[V], beta[V];
  weights_of<WT, V>(a.gamma, e, 1.0f, gamma);
  weights_of<WT, V>(a.beta, e, 0.0f, beta);
  int group[V];
#pragma unroll
  for (int k = 0; k < V; ++k) group[k] = p.on ? (int)fdiv((uint32_t)(p.col * V + k), a.div_Cg) : 0;
  const int turns = p.on && p.r < a.S ? (a.S - p.r + p.RB - 1) / p.RB : 0;
  const float inv = 1.0f / ((float)a.S * (float)a.Cg);
  // sums about a first mean, then its rounding error taken out
  float s[1][V], d2[2][V], mean[V];
#pragma unroll
  for (int k = 0; k < V; ++k) s[0][k] = d2[0][k] = d2[1][k] = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (j >= turns) continue;
    float f[V];
    unpack<DT, 16>(v[j], f);
#pragma unroll
    for (int k = 0; k < V; ++k) s[0][k] += f[k];
  }
  group_sums<1, V, kHeldThreads>(a.sg, group, s, lds, sums[0]);
#pragma unroll
  for (int k = 0; k < V; ++k) mean[k] = sums[0][0][group[k]] * inv;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (j >= turns) continue;
    float f[V];
    unpack<DT, 16>(v[j], f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float d = f[k] - mean[k];
      d2[0][k] += d;
      d2[1][k] = __builtin_fmaf(d, d, d2[1][k]);
    }
  }
  group_sums<2, V, kHeldThreads>(a.sg, group, d2, lds, sums[1]);
  if ((int)threadIdx.x < a.sg) { // this thread's group is its own number
    const float e1 = sums[1][0][threadIdx.x] * inv, off = sums[1][1][threadIdx.x] * inv - e1 * e1;
    const float r = 1.0f / sqrtf((off < 0.0f ? 0.0f : off) + a.eps); // (NaN stays)
    sums[2][0][threadIdx.x] = e1;
    sums[2][1][threadIdx.x] = r;
    float *to = a.stats + ((int64_t)p.n * a.G + (int)fdiv((uint32_t)p.c0, a.div_Cg) + threadIdx.x) * 3;
    to[0] = sums[0][0][threadIdx.x] * inv;
    to[1] = e1;
    to[2] = r;
  }
  __syncthreads();
  float rest[V], r[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    rest[k] = sums[2][0][group[k]];
    r[k] = sums[2][1][group[k]];
  }
  const int64_t to = p.n * a.sout.n + (int64_t)p.r * a.sout.s + e;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (j >= turns) continue;
    float f[V];
    unpack<DT, 16>(v[j], f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float z = __builtin_fmaf(((f[k] - mean[k]) - rest[k]) * r[k], gamma[k], beta[k]);
      f[k] = SILU ? z * logistic(z) : z;
    }
    store_part<DT>(a.out, to + (int64_t)j * p.RB * a.sout.s, V, pack<DT, 16>(f));
  }
}

template <int DT, int WT, bool SILU>
__global__ __launch_bounds__(kHeldBackThreads) void held_gradient_kernel(const ChanArgs a) {
  constexpr int V = kVec<DT>, NV = kHeldBackVectors, THREADS = kHeldBackThreads, STRIDE = THREADS * V;
  __shared__ float part[2 * STRIDE]; // sums of g and of g h by channel and position of a turn
  __shared__ float lds[2][8][THREADS / 64], sums[2][8];
  const Held p = Held::of<THREADS>(a);
  const int e = p.c0 + (p.on ? p.col * V : 0), row = p.on ? p.r : 0;
  Vec<16> v[NV], w[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) { // (positions past the end: the last one, left out below)
    const int64_t at = min(row + j * p.RB, a.S - 1);
    v[j] = load_part<DT>(a.x, p.n * a.sx.n + at * a.sx.s + e, V);
    w[j] = load_part<DT>(a.dy, p.n * a.sdy.n + at * a.sdy.s + e, V);
  }
  Channels<DT, WT> ch;
  ch.load(a, p.n, e);
  int group[V];
#pragma unroll
  for (int k = 0; k < V; ++k) group[k] = p.on ? (int)fdiv((uint32_t)(p.col * V + k), a.div_Cg) : 0;
  const int turns = p.on && p.r < a.S ? (a.S - p.r + p.RB - 1) / p.RB : 0;
  float by[2][V];
#pragma unroll
  for (int k = 0; k < V; ++k) by[0][k] = by[1][k] = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (j >= turns) continue;
    float g[V], h[V];
    gradient_of<DT, WT, SILU>(ch, v[j], w[j], g, h);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      by[0][k] += g[k];
      by[1][k] = __builtin_fmaf(g[k], h[k], by[1][k]);
    }
  }
  const bool wanted = a.dgamma || a.dbeta;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (wanted && p.on) {
      part[(p.col * V + k) * p.RB + p.r] = by[0][k];
      part[STRIDE + (p.col * V + k) * p.RB + p.r] = by[1][k];
    }
    by[0][k] *= ch.gamma[k];
    by[1][k] *= ch.gamma[k];
  }
  group_sums<2, V, THREADS>(a.sg, group, by, lds, sums);
  const float inv = 1.0f / ((float)a.S * (float)a.Cg);
  float mg[V], mh[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    mg[k] = sums[0][group[k]] * inv;
    mh[k] = sums[1][group[k]] * inv;
  }
  const int64_t to = p.n * a.sout.n + (int64_t)p.r * a.sout.s + e;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (j >= turns) continue;
    float g[V], h[V];
    gradient_of<DT, WT, SILU>(ch, v[j], w[j], g, h);
#pragma unroll
    for (int k = 0; k < V; ++k) g[k] = ch.r[k] * (__builtin_fmaf(g[k], ch.gamma[k], -mg[k]) - h[k] * mh[k]);
    store_part<DT>(a.out, to + (int64_t)j * p.RB * a.sout.s, V, pack<DT, 16>(g));
  }
  if (!wanted) return;
  // the weights' gradients by channel (a wave to one): of a single sample, or its part
  const int lane = threadIdx.x & 63;
  for (int c = threadIdx.x >> 6; c < a.CS; c += THREADS / 64) {
    float s = 0.0f, t = 0.0f;
    for (int i = lane; i < p.RB; i += 64) {
      s += part[c * p.RB + i];
      t += part[STRIDE + c * p.RB + i];
    }
    s = lanes_sum<64>(s);
    t = lanes_sum<64>(t);
    if (lane != 0) continue;
    const int at = p.c0 + c;
    if (a.N == 1) {
      typedef typename El<WT>::bits bits;
      if (a.dbeta) ((bits *)a.dbeta)[at] = (bits)narrow<WT>(s);
      if (a.dgamma) ((bits *)a.dgamma)[at] = (bits)narrow<WT>(t);
    } else {
      a.part[(int64_t)p.n * 2 * a.C + at] = s;
      a.part[(int64_t)p.n * 2 * a.C + a.C + at] = t;
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
// The pass that writes goes backwards, so that it begins with what the first pass
// read last and the caches still hold.
ChanArgs backwards(ChanArgs a) {
  a.chunk = a.apply_chunk;
  a.chunks = a.apply_chunks;
  a.div_chunks = make_fastdiv((uint32_t)a.chunks);
  a.last = (uint32_t)((int64_t)a.N * a.chunks * a.slabs - 1);
  return a;
}

template <int DT, int WT, Cover C, bool SILU> hipError_t forward(const ChanArgs &a, hipStream_t st) {
  const dim3 block(kChanThreads);
  if constexpr (C == WHOLE) {
    if (a.sg) {
      hipLaunchKernelGGL((held_kernel<DT, WT, SILU>), dim3((unsigned)(a.N * (a.G / a.sg))), dim3(kHeldThreads), 0, st, a);
      return hipGetLastError();
    }
  }
  over_blocks(a, [&](const ChanArgs &b, dim3 grid) { hipLaunchKernelGGL((stats_kernel<DT, C>), grid, block, 0, st, b); });
  hipLaunchKernelGGL((merge_kernel<DT>), dim3((unsigned)(a.N * a.G)), dim3(kMergeThreads), 0, st, a);
  over_blocks(backwards(a), [&](const ChanArgs &b, dim3 grid) {
    if (a.far) hipLaunchKernelGGL((apply_kernel<DT, WT, C, SILU, true>), grid, block, 0, st, b);
    else hipLaunchKernelGGL((apply_kernel<DT, WT, C, SILU, false>), grid, block, 0, st, b);
  });
  return hipGetLastError();
}

template <int DT, int WT, Cover C, bool SILU> hipError_t backward(const ChanArgs &a, hipStream_t st) {
  const dim3 block(kChanThreads);
  const unsigned columns = a.dgamma || a.dbeta ? (a.C + 63) / 64 : 0;
  if constexpr (C == WHOLE) {
    if (a.sg) {
      hipLaunchKernelGGL((held_gradient_kernel<DT, WT, SILU>), dim3((unsigned)(a.N * (a.G / a.sg))),
                         dim3(kHeldBackThreads), 0, st, a);
      if (a.N > 1 && columns) {
        ChanArgs b = a;
        b.G = 0; // (no groups to gather: channels alone)
        hipLaunchKernelGGL((gather_kernel<WT>), dim3(columns), dim3(kMergeThreads), 0, st, b);
      }
      return hipGetLastError();
    }
  }
  over_blocks(a, [&](const ChanArgs &b, dim3 grid) {
    hipLaunchKernelGGL((sums_kernel<DT, WT, C, SILU>), grid, block, 0, st, b);
  });
  if (a.N * a.G + columns)
    hipLaunchKernelGGL((gather_kernel<WT>), dim3((unsigned)(a.N * a.G) + columns), dim3(kMergeThreads), 0, st, a);
  if (a.N)
    over_blocks(backwards(a), [&](const ChanArgs &b, dim3 grid) {
      if (a.far) hipLaunchKernelGGL((gradient_kernel<DT, WT, C, SILU, true>), grid, block, 0, st, b);
      else hipLaunchKernelGGL((gradient_kernel<DT, WT, C, SILU, false>), grid, block, 0, st, b);
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
