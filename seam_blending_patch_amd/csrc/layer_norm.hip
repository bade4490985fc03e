// layer_norm.hip -- layer norm, forward and backward, gfx950.
//
// Rows of D elements: m = sum x / D, v = sum (x - m)^2 / D,
// r = 1 / sqrt(v + eps), h = (x - m) r, y = h gamma + beta.  With
// g = dy gamma the gradient is
//   dx = r (g - mean(g) - h mean(g h)),
//   dgamma = sum over rows of dy h,  dbeta = sum over rows of dy.
//
// Statistics are fp32 and corrected two-pass: m0 = sum x / D rounded, then
// over d = x - m0 both e = sum d / D and sum d^2, so that v = sum d^2 / D - e^2
// and x - m = d - e.  e is of the size of m0's rounding error, so nothing
// cancels, and a mean that is large against the spread costs no accuracy.
// The backward pass forms the statistics again from the rows it reads anyway:
// nothing has to be kept from the forward pass.

#include "sb_row.h"
#include "sb_transformer.h"

#include <algorithm>
#include <type_traits>

namespace sb {

__device__ __forceinline__ int64_t row_offset(uint32_t row, const FastDiv &inner, const RowStride &s) {
  const uint32_t o = fdiv(row, inner);
  return (int64_t)o * s.o + (int64_t)(row - o * inner.d) * s.i;
}

// ---------------------------------------------------------------------------
// Rows that fit the registers of LANES threads, NV vectors each: every element
// is read once.  A block of 256 threads (or LANES, if more) takes as many rows
// as it has groups of LANES.
// ---------------------------------------------------------------------------
template <int LANES> constexpr int kRowThreads = LANES > kLNThreads ? LANES : kLNThreads;
// Row lengths that have a kernel whose stores pass the caches, for outputs that
// those could not hold (a branch at the store instead loses what it gains).
template <int LANES> constexpr bool kFarRows = LANES >= 64;

// A thread's vector u holds the elements of its row from (u * LANES + lane) * V
// on.  NV is never more than the row needs, so only the last one can pass the
// row's end, and be cut by it where the row is no whole number of vectors (TAIL).
template <int NV, bool TAIL> constexpr Cover cover(int u) { return u < NV - 1 ? WHOLE : TAIL ? CUT : WHOLE_OR_NONE; }
// f<u>() for every u below NV
template <int NV, class F, int U = 0> __device__ __forceinline__ void each(F f) {
  if constexpr (U < NV) {
    f(std::integral_constant<int, U>());
    each<NV, F, U + 1>(f);
  }
}

// x as fp32 -> d = x - m0 in place, zero where the row has no element
template <int DT, int LANES, int NV, bool TAIL>
__device__ __forceinline__ void subtract(float (&x)[NV][kVec<DT>], float m0, int lane, int D) {
  constexpr int V = kVec<DT>;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int e = (u * LANES + lane) * V;
#pragma unroll
    for (int k = 0; k < V; ++k) x[u][k] = u < NV - 1 || (TAIL ? e + k < D : e < D) ? x[u][k] - m0 : 0.f;
  }
}

// Rows that a group works on together: two where a row is a single vector of a
// thread, so that one fills what the other waits for (243360 rows of 128 bf16:
// one 26.0 us, two 23.8, four 24.5).
template <int LANES, int NV> constexpr int kRowsTogether = NV == 1 && LANES <= 64 ? 2 : 1;
// Whether gamma and beta are requested beside the row, not after its sums: up to
// 24 elements a thread (65536 x 512 bf16 26.2 -> 23.4 us, 131072 x 1536 148 ->
// 144; with 32 elements 65536 x 2048 fp16 100 -> 113), and not where a block of
// 1024 has one row (4096 x 16384 73 -> 78).
template <int LANES, int ELEMENTS> constexpr bool kWeightsEarly = ELEMENTS <= 24 && LANES <= 256;

// Forward.  Bound by the copy of the rows: 65536 x 2048 fp16, 537 MB in 98 us
// (5.5 TB/s, a large copy's rate 5.2), 20280 x 12 heads of 128 bf16 out of a
// packed projection, 125 MB in 23.4 us (5.3 TB/s), 20280 x 1536 bf16 in 20.5 us
// (within the last-level cache).  A wave to a row up to 256 vectors: no barrier.
template <int DT, int WDT, int LANES, int NV, bool TAIL, bool NT = false>
__global__ __launch_bounds__(kRowThreads<LANES>) void ln_row_kernel(const LNArgs A) {
  constexpr int V = kVec<DT>, GROUPS = kRowThreads<LANES> / LANES, R = kRowsTogether<LANES, NV>;
  __shared__ float lds[2][LANES > 64 ? 2 * kRowThreads<LANES> / 64 : 1];
  int turn = 0;
  const int lane = threadIdx.x % LANES;
  for (int64_t r0 = (int64_t)blockIdx.x * GROUPS * R; r0 < A.rows; r0 += (int64_t)gridDim.x * GROUPS * R) {
    const int64_t row = r0 + threadIdx.x / LANES; // and R - 1 more, GROUPS apart
    Vec<16> raw[R][NV];
    float x[R][NV][V], s1[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      // every lane takes part in the sums
      const int64_t xo = row_offset((uint32_t)min(row + i * GROUPS, A.rows - 1), A.inner, A.sx);
      each<NV>([&](auto u) { raw[i][u] = request_row<DT, cover<NV, TAIL>(u)>(A.x, xo, (u * LANES + lane) * V, A.D); });
    }
    constexpr bool EARLY = kWeightsEarly<LANES, NV * V>;
    float w[NV][V], b[NV][V];
    auto weights = [&](auto u) {
      const int c = (u * LANES + lane) * V;
      if (A.gamma) load_weights<WDT, V, cover<NV, TAIL>(u)>(A.gamma, c, A.D, w[u]);
      if (A.beta) load_weights<WDT, V, cover<NV, TAIL>(u)>(A.beta, c, A.D, b[u]);
    };
    if (EARLY) each<NV>(weights);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s1[i] = 0.f;
      each<NV>([&](auto u) {
        settle_row<DT, cover<NV, TAIL>(u)>(raw[i][u], (u * LANES + lane) * V, A.D);
        unpack<DT, 16>(raw[i][u], x[i][u]);
      });
#pragma unroll
      for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int k = 0; k < V; ++k) s1[i] += x[i][u][k];
    }
    group_sum<LANES>(s1, lds, turn);
    float s[2 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      subtract<DT, LANES, NV, TAIL>(x[i], s1[i] * A.inv_d, lane, A.D);
      s[2 * i] = s[2 * i + 1] = 0.f;
#pragma unroll
      for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          s[2 * i] += x[i][u][k];
          s[2 * i + 1] = fmaf(x[i][u][k], x[i][u][k], s[2 * i + 1]);
        }
    }
    group_sum<LANES>(s, lds, turn);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float e = s[2 * i] * A.inv_d;
      const float r = 1.0f / sqrtf(fmaxf(fmaf(s[2 * i + 1], A.inv_d, -e * e), 0.f) + A.eps);
      if (row + i * GROUPS >= A.rows) break;
      const int64_t yo = row_offset((uint32_t)(row + i * GROUPS), A.inner, A.sout);
      each<NV>([&](auto u) {
        if (!EARLY) weights(u);
#pragma unroll
        for (int k = 0; k < V; ++k)
          x[i][u][k] = fmaf((x[i][u][k] - e) * r, A.gamma ? w[u][k] : 1.f, A.beta ? b[u][k] : 0.f);
        store_row<DT, cover<NV, TAIL>(u), NT>(A.out, yo, (u * LANES + lane) * V, A.D, pack<DT, 16>(x[i][u]));
      });
    }
  }
}

// the total of float i of the blocks of partials, to where it belongs
template <int WDT, int LANES, int V> __device__ __forceinline__ void store_column(const LNArgs &A, int64_t i, float t) {
  const bool beta = i >= A.cols;
  const uint32_t j = (uint32_t)(beta ? i - A.cols : i);
  const uint32_t u = j / (LANES * V), k = j / LANES % V, l = j % LANES;
  const int64_t col = ((int64_t)u * LANES + l) * V + k;
  void *out = beta ? A.dbeta : A.dgamma;
  if (out && col < A.D) ((typename El<WDT>::bits *)out)[col] = (typename El<WDT>::bits)narrow<WDT>(t);
}

// dx and the columns' sums in one pass over x and dy.  A block keeps taking
// rows, a thread the same columns of each, so dgamma and dbeta add up in
// registers; at the end the block's rows are merged and written as one block of
// partials.  (Requesting the next row before this one is used costs more in
// registers than it hides: 32768 x 4096 bf16 147 -> 173 us, 8192 x 16384 189 ->
// 228, spilled.)
// Bound by the three rows it moves: 65536 x 2048 fp16, 805 MB in 144-151 us
// (5.3-5.6 TB/s, a large copy's rate 5.2) and 5 us for the reduction; 20280 x
// 1536 bf16, 187 MB in 34.7 and 4.8 us.  (LNLayout has the layouts measured.)
template <int DT, int WDT, int LANES, int NV, bool TAIL, bool NT = false>
__global__ __launch_bounds__(kRowThreads<LANES>) void ln_backward_kernel(const LNArgs A) {
  constexpr int V = kVec<DT>, T = kRowThreads<LANES>, GROUPS = T / LANES, COLS = LANES * NV * V;
  // partials to merge: one of each wave, or of each group where that is wider
  constexpr int COPIES = LANES < 64 ? T / 64 : GROUPS;
  __shared__ float lds[2][LANES > 64 ? 4 * T / 64 : 1];
  __shared__ float merge[COPIES > 1 ? COPIES * COLS : 1];
  int turn = 0;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  float w[NV][V], dg[NV][V], db[NV][V];
  each<NV>([&](auto u) {
    if (A.gamma) load_weights<WDT, V, cover<NV, TAIL>(u)>(A.gamma, (u * LANES + lane) * V, A.D, w[u]);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (!A.gamma) w[u][k] = 1.f;
      dg[u][k] = db[u][k] = 0.f;
    }
  });
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < A.rows; r0 += step) {
    const int64_t row = r0 + group;
    const uint32_t at = (uint32_t)min(row, A.rows - 1); // every lane takes part in the sums
    const int64_t xo = row_offset(at, A.inner, A.sx), go = row_offset(at, A.inner, A.sdy);
    Vec<16> xr[NV], gr[NV];
    each<NV>([&](auto u) {
      xr[u] = request_row<DT, cover<NV, TAIL>(u)>(A.x, xo, (u * LANES + lane) * V, A.D);
      gr[u] = request_row<DT, cover<NV, TAIL>(u)>(A.dy, go, (u * LANES + lane) * V, A.D);
    });
    float x[NV][V], g[NV][V];
    each<NV>([&](auto u) {
      settle_row<DT, cover<NV, TAIL>(u)>(xr[u], (u * LANES + lane) * V, A.D);
      settle_row<DT, cover<NV, TAIL>(u)>(gr[u], (u * LANES + lane) * V, A.D);
      unpack<DT, 16>(xr[u], x[u]);
      unpack<DT, 16>(gr[u], g[u]);
    });
    if (row >= A.rows) { // an absent row adds nothing
#pragma unroll
      for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int k = 0; k < V; ++k) x[u][k] = g[u][k] = 0.f;
    }
    float s1[1] = {0.f};
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int k = 0; k < V; ++k) s1[0] += x[u][k];
    group_sum<LANES>(s1, lds, turn);
    subtract<DT, LANES, NV, TAIL>(x, s1[0] * A.inv_d, lane, A.D);
    float s[4] = {0.f, 0.f, 0.f, 0.f}; // of d, d^2, g, g d
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float gw = g[u][k] * w[u][k];
        s[0] += x[u][k];
        s[1] = fmaf(x[u][k], x[u][k], s[1]);
        s[2] += gw;
        s[3] = fmaf(gw, x[u][k], s[3]);
      }
    group_sum<LANES>(s, lds, turn);
    const float e = s[0] * A.inv_d, mg = s[2] * A.inv_d;
    float r = 1.0f / sqrtf(fmaxf(fmaf(s[1], A.inv_d, -e * e), 0.f) + A.eps);
    const float mgh = r * fmaf(s[3], A.inv_d, -e * mg);
    if (row >= A.rows) r = 0.f; // nor where eps is 0
    const int64_t yo = row < A.rows ? row_offset((uint32_t)row, A.inner, A.sout) : 0;
    each<NV>([&](auto u) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float h = (x[u][k] - e) * r;
        dg[u][k] = fmaf(g[u][k], h, dg[u][k]);
        db[u][k] += g[u][k];
        x[u][k] = r * (fmaf(-h, mgh, g[u][k] * w[u][k]) - mg);
      }
      if (row < A.rows)
        store_row<DT, cover<NV, TAIL>(u), NT>(A.out, yo, (u * LANES + lane) * V, A.D, pack<DT, 16>(x[u]));
    });
  }
  if (!A.part) return;
  // Columns in the order [u][k][lane], so that a wave's stores are contiguous.
  // A single block's sums are the weights' gradients themselves.
  const bool alone = gridDim.x == 1;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float *part = A.part + ((int64_t)blockIdx.x * 2 + which) * COLS;
    auto put = [&](int i, float t) {
      if (alone) store_column<WDT, LANES, V>(A, which * COLS + i, t);
      else part[i] = t;
    };
    auto &v = which ? db : dg;
    if constexpr (COPIES == 1) {
#pragma unroll
      for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int k = 0; k < V; ++k) put((u * V + k) * LANES + lane, v[u][k]);
    } else {
      if (which) __syncthreads();
#pragma unroll
      for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          float t = v[u][k];
#pragma unroll
          for (int o = LANES; o < 64; o <<= 1) t += __shfl_xor(t, o);
          if (LANES >= 64 || (threadIdx.x & 63) < LANES)
            merge[(LANES < 64 ? threadIdx.x / 64 : group) * COLS + (u * V + k) * LANES + lane] = t;
        }
      __syncthreads();
      for (int i = threadIdx.x; i < COLS; i += T) {
        float t = merge[i];
#pragma unroll
        for (int c = 1; c < COPIES; ++c) t += merge[c * COLS + i];
        put(i, t);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Longer rows: split into chunks that fit a block's registers, however few rows
// there are.  A chunk's statistics are corrected two-pass about its own m0;
// a row's are merged from its chunks' (Chan, Golub & LeVeque), about the first
// chunk's m0, called K: with a chunk's mean K + delta,
//   E = sum n delta / D,  M2 = sum (M2_c + n (delta - E)^2),  x - m = (x - K) - E.
// 4 rows of 798720 bf16: 14 us forward, 35 backward with its reduction (a block
// of 1024 threads to a row: 178 and 435); 1000 rows of 40000: 49 and 100 (54 and
// 108), of which reading the rows twice is the bound.
// ---------------------------------------------------------------------------
template <int DT> constexpr int kChunk = kLNThreads * kChunkVectors * kVec<DT>;
struct ChunkStat { // 8 floats of workspace
  float m0, e, m2, g, gd; // mean m0 + e, squares about it, sums of g and g (x - m0)
  float unused[3];
};

// one block a chunk (blockIdx.x) of every gridDim.y-th row
template <int DT, int WDT, bool BACKWARD> __global__ __launch_bounds__(kLNThreads) void ln_chunk_kernel(const LNArgs A) {
  constexpr int V = kVec<DT>, NV = kChunkVectors, SUMS = BACKWARD ? 4 : 2;
  __shared__ float lds[2][SUMS * kLNThreads / 64];
  int turn = 0;
  const int c0 = blockIdx.x * kChunk<DT> + threadIdx.x * V, here = min(kChunk<DT>, A.D - (int)blockIdx.x * kChunk<DT>);
  for (int64_t row = blockIdx.y; row < A.rows; row += gridDim.y) {
    const int64_t xo = row_offset((uint32_t)row, A.inner, A.sx);
    float x[NV][V], g[NV][V], s1[1] = {0.f};
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = c0 + u * kLNThreads * V;
      load_floats<DT, V>(A.x, xo + c, A.D - c, x[u]);
    }
    if constexpr (BACKWARD) {
      const int64_t go = row_offset((uint32_t)row, A.inner, A.sdy);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int c = c0 + u * kLNThreads * V;
        load_floats<DT, V>(A.dy, go + c, A.D - c, g[u]);
        if (A.gamma) {
          float w[V];
          load_floats<WDT, V>(A.gamma, c, A.D - c, w);
#pragma unroll
          for (int k = 0; k < V; ++k) g[u][k] *= w[k];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int k = 0; k < V; ++k) s1[0] += x[u][k];
    group_sum<kLNThreads>(s1, lds, turn);
    const float m0 = s1[0] / (float)here;
    float s[SUMS] = {};
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float d = c0 + u * kLNThreads * V + k < A.D ? x[u][k] - m0 : 0.f;
        s[0] += d;
        s[1] = fmaf(d, d, s[1]);
        if constexpr (BACKWARD) {
          s[SUMS - 2] += g[u][k];
          s[SUMS - 1] = fmaf(g[u][k], d, s[SUMS - 1]);
        }
      }
    group_sum<kLNThreads>(s, lds, turn);
    if (threadIdx.x == 0) {
      const float e = s[0] / (float)here;
      ChunkStat *st = reinterpret_cast<ChunkStat *>(A.chunks) + row * gridDim.x + blockIdx.x;
      st->m0 = m0;
      st->e = e;
      st->m2 = fmaf(-e, s[0], s[1]);
      if constexpr (BACKWARD) {
        st->g = s[SUMS - 2];
        st->gd = s[SUMS - 1];
      }
    }
  }
}

// a row's statistics from its chunks': (K, E, r, mean of g) and the mean of g h
template <int DT, bool BACKWARD> __global__ __launch_bounds__(kLNThreads) void ln_merge_kernel(const LNArgs A, int chunks) {
  constexpr int SUMS = BACKWARD ? 3 : 1;
  __shared__ float lds[2][SUMS * kLNThreads / 64];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
    const ChunkStat *st = reinterpret_cast<const ChunkStat *>(A.chunks) + row * chunks;
    const float K = st[0].m0;
    float s1[1] = {0.f};
    for (int c = threadIdx.x; c < chunks; c += kLNThreads)
      s1[0] = fmaf((float)min(kChunk<DT>, A.D - c * kChunk<DT>), (st[c].m0 - K) + st[c].e, s1[0]);
    group_sum<kLNThreads>(s1, lds, turn);
    const float E = s1[0] * A.inv_d;
    float s[SUMS] = {};
    for (int c = threadIdx.x; c < chunks; c += kLNThreads) {
      const float off = (st[c].m0 - K) - E, d = off + st[c].e;
      s[0] += fmaf((float)min(kChunk<DT>, A.D - c * kChunk<DT>) * d, d, st[c].m2);
      if constexpr (BACKWARD) {
        s[SUMS - 2] += st[c].g;
        s[SUMS - 1] += fmaf(st[c].g, off, st[c].gd); // g (x - m), x - m = (x - m0) + off
      }
    }
    group_sum<kLNThreads>(s, lds, turn);
    if (threadIdx.x == 0) {
      const float r = 1.0f / sqrtf(fmaxf(s[0] * A.inv_d, 0.f) + A.eps);
      const float mg = BACKWARD ? s[SUMS - 2] * A.inv_d : 0.f;
      reinterpret_cast<float4 *>(A.rowstat)[2 * row] = make_float4(K, E, r, mg);
      if constexpr (BACKWARD) A.rowstat[8 * row + 4] = r * s[SUMS - 1] * A.inv_d;
    }
  }
}

// y: a block has 256 vectors of columns (blockIdx.x) and every gridDim.y-th row
template <int DT, int WDT> __global__ __launch_bounds__(kLNThreads) void ln_apply_kernel(const LNArgs A) {
  constexpr int V = kVec<DT>;
  const int c = (blockIdx.x * kLNThreads + threadIdx.x) * V;
  float w[V], b[V];
#pragma unroll
  for (int k = 0; k < V; ++k) w[k] = 1.f, b[k] = 0.f;
  if (A.gamma) load_floats<WDT, V>(A.gamma, c, A.D - c, w);
  if (A.beta) load_floats<WDT, V>(A.beta, c, A.D - c, b);
  for (int64_t row = blockIdx.y; row < A.rows; row += gridDim.y) {
    const float4 st = reinterpret_cast<const float4 *>(A.rowstat)[2 * row];
    float x[V];
    load_floats<DT, V>(A.x, row_offset((uint32_t)row, A.inner, A.sx) + c, A.D - c, x);
#pragma unroll
    for (int k = 0; k < V; ++k) x[k] = fmaf(((x[k] - st.x) - st.y) * st.z, w[k], b[k]);
    store_part<DT>(A.out, row_offset((uint32_t)row, A.inner, A.sout) + c, A.D - c, pack<DT, 16>(x));
  }
}

// dx and the column sums: a block has 256 vectors of columns (blockIdx.x) and
// every gridDim.y-th row
template <int DT, int WDT>
__global__ __launch_bounds__(kLNThreads) void ln_columns_kernel(const LNArgs A) {
  constexpr int V = kVec<DT>;
  const int c = (blockIdx.x * kLNThreads + threadIdx.x) * V;
  float w[V], dg[V], db[V];
#pragma unroll
  for (int k = 0; k < V; ++k) w[k] = 1.f, dg[k] = db[k] = 0.f;
  if (A.gamma) load_floats<WDT, V>(A.gamma, c, A.D - c, w);
  for (int64_t row = blockIdx.y; row < A.rows; row += gridDim.y) {
    const float4 st = reinterpret_cast<const float4 *>(A.rowstat)[2 * row];
    const float mgh = A.rowstat[8 * row + 4];
    float x[V], g[V];
    load_floats<DT, V>(A.x, row_offset((uint32_t)row, A.inner, A.sx) + c, A.D - c, x);
    load_floats<DT, V>(A.dy, row_offset((uint32_t)row, A.inner, A.sdy) + c, A.D - c, g);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float h = ((x[k] - st.x) - st.y) * st.z;
      dg[k] = fmaf(g[k], h, dg[k]);
      db[k] += g[k];
      x[k] = st.z * (fmaf(-h, mgh, g[k] * w[k]) - st.w);
    }
    store_part<DT>(A.out, row_offset((uint32_t)row, A.inner, A.sout) + c, A.D - c, pack<DT, 16>(x));
  }
  if (A.part) {
    // floats of a block of partials: columns in the order [u][k][thread], so
    // that stores of a wave are contiguous
    float *p = A.part + (int64_t)blockIdx.y * 2 * A.cols + (int64_t)blockIdx.x * kLNThreads * V + threadIdx.x;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      p[k * kLNThreads] = dg[k];
      p[A.cols + k * kLNThreads] = db[k];
    }
  }
}

// dgamma and dbeta: the partials' sums, in a fixed order.  A block takes 16
// floats of a block of partials (of 2 * cols), as 4 vectors; its 256 groups of
// 4 threads take every 256th block of partials each, so that a thousand of
// them are four loads deep and a thousand columns are 128 blocks wide.
constexpr int kReduceThreads = 1024, kReduceCols = 16;
template <int WDT, int LANES, int V>
__global__ __launch_bounds__(kReduceThreads) void ln_reduce_kernel(const LNArgs A) {
  static_assert(LANES * V % kReduceCols == 0, "cols is a multiple of kReduceCols");
  __shared__ float lds[kReduceThreads / 64][kReduceCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, quad = threadIdx.x & 3;
  const float4 *p = reinterpret_cast<const float4 *>(A.part + (int64_t)blockIdx.x * kReduceCols) + quad;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int b = threadIdx.x >> 2; b < A.nparts; b += kReduceThreads / 4) {
    const float4 v = p[(int64_t)b * 2 * A.cols / 4];
    s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int o = 4; o < 64; o <<= 1) s[k] += __shfl_xor(s[k], o);
    if (lane < 4) lds[wave][quad * 4 + k] = s[k];
  }
  __syncthreads();
  if (threadIdx.x < kReduceCols) {
    float t = lds[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kReduceThreads / 64; ++w) t += lds[w][threadIdx.x];
    store_column<WDT, LANES, V>(A, (int64_t)blockIdx.x * kReduceCols + threadIdx.x, t);
  }
}

// the same where there are columns enough to fill the chip: a thread a column
template <int WDT, int LANES, int V>
__global__ __launch_bounds__(kLNThreads) void ln_reduce_columns_kernel(const LNArgs A) {
  const int64_t i = (int64_t)blockIdx.x * kLNThreads + threadIdx.x;
  if (i >= 2 * (int64_t)A.cols) return;
  float t = 0.f;
#pragma unroll 4
  for (int b = 0; b < A.nparts; ++b) t += A.part[(int64_t)b * 2 * A.cols + i];
  store_column<WDT, LANES, V>(A, i, t);
}

template <int DT, int WDT, int LANES, int NV> hipError_t launch_rows(const LNArgs &a, hipStream_t st) {
  constexpr int T = kRowThreads<LANES>, ROWS = T / LANES * kRowsTogether<LANES, NV>; // of a block
  const unsigned blocks = (unsigned)std::min<int64_t>((a.rows + ROWS - 1) / ROWS, kMaxBlocksX / (T / kLNThreads));
  const auto kernel = a.D % kVec<DT>               ? ln_row_kernel<DT, WDT, LANES, NV, true>
                      : kFarRows<LANES> && a.far ? ln_row_kernel<DT, WDT, LANES, NV, false, kFarRows<LANES>>
                                                 : ln_row_kernel<DT, WDT, LANES, NV, false>;
  hipLaunchKernelGGL(kernel, dim3(blocks), dim3(T), 0, st, a);
  return hipGetLastError();
}

// of rows split into chunks, to A.rowstat
template <int DT, int WDT, bool BACKWARD> hipError_t launch_statistics(const LNArgs &a, hipStream_t st) {
  const int chunks = (a.D + kChunk<DT> - 1) / kChunk<DT>;
  hipLaunchKernelGGL((ln_chunk_kernel<DT, WDT, BACKWARD>), dim3((unsigned)chunks, (unsigned)std::min<int64_t>(a.rows, kMaxGridY)),
                     dim3(kLNThreads), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((ln_merge_kernel<DT, BACKWARD>), dim3((unsigned)std::min<int64_t>(a.rows, kMaxBlocksX)),
                     dim3(kLNThreads), 0, st, a, chunks);
  return hipGetLastError();
}

template <int DT, int WDT> hipError_t launch_forward(const LNArgs &a, hipStream_t st) {
  const int nv = (a.D + kVec<DT> - 1) / kVec<DT>; // vectors of a row
  if (nv <= 4) return launch_rows<DT, WDT, 4, 1>(a, st);
  if (nv <= 8) return launch_rows<DT, WDT, 8, 1>(a, st);
  if (nv <= 16) return launch_rows<DT, WDT, 16, 1>(a, st);
  if (nv <= 32) return launch_rows<DT, WDT, 32, 1>(a, st);
  if (nv <= 64) return launch_rows<DT, WDT, 64, 1>(a, st);
  if (nv <= 128) return launch_rows<DT, WDT, 64, 2>(a, st);
  if (nv <= 192) return launch_rows<DT, WDT, 64, 3>(a, st);
  if (nv <= 256) return launch_rows<DT, WDT, 64, 4>(a, st);
  if (nv <= 512) return launch_rows<DT, WDT, 256, 2>(a, st);
  if (nv <= 768) return launch_rows<DT, WDT, 256, 3>(a, st);
  if (nv <= 1024) return launch_rows<DT, WDT, 256, 4>(a, st);
  if (nv <= 2048) return launch_rows<DT, WDT, 1024, 2>(a, st);
  if (nv <= 3072) return launch_rows<DT, WDT, 1024, 3>(a, st);
  if (nv <= kForwardVectors) return launch_rows<DT, WDT, 1024, 4>(a, st);
  const hipError_t e = launch_statistics<DT, WDT, false>(a, st);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((nv + kLNThreads - 1) / kLNThreads), (unsigned)std::min<int64_t>(a.rows, 1024));
  hipLaunchKernelGGL((ln_apply_kernel<DT, WDT>), grid, dim3(kLNThreads), 0, st, a);
  return hipGetLastError();
}

template <int WDT, int LANES, int V> hipError_t launch_reduce(const LNArgs &a, hipStream_t st) {
  if (!a.part) return hipSuccess;
  // (40960 columns and 51 blocks of partials: 6.9 us by columns, 19 by blocks of
  // 16; 16384 and 256 of them 12.9 by blocks)
  if (a.cols >= 32768) {
    hipLaunchKernelGGL((ln_reduce_columns_kernel<WDT, LANES, V>),
                       dim3((unsigned)((2 * (int64_t)a.cols + kLNThreads - 1) / kLNThreads)), dim3(kLNThreads), 0, st, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((ln_reduce_kernel<WDT, LANES, V>), dim3((unsigned)(2 * (int64_t)a.cols / kReduceCols)),
                     dim3(kReduceThreads), 0, st, a);
  return hipGetLastError();
}

template <int DT, int WDT, int LANES, int NV> hipError_t launch_backward_rows(const LNArgs &a, hipStream_t st) {
  constexpr int T = kRowThreads<LANES>;
  if (a.nparts > 0) {
    const auto kernel = a.D % kVec<DT>               ? ln_backward_kernel<DT, WDT, LANES, NV, true>
                        : kFarRows<LANES> && a.far ? ln_backward_kernel<DT, WDT, LANES, NV, false, kFarRows<LANES>>
                                                   : ln_backward_kernel<DT, WDT, LANES, NV, false>;
    hipLaunchKernelGGL(kernel, dim3(a.nparts), dim3(T), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.nparts == 1) return e;
  }
  return launch_reduce<WDT, LANES, kVec<DT>>(a, st);
}

template <int DT, int WDT> hipError_t launch_backward(const LNArgs &a, hipStream_t st) {
  constexpr int V = kVec<DT>;
  const LNLayout lay = backward_layout((a.D + V - 1) / V);
  switch (lay.lanes * 16 + lay.nv) {
  case 4 * 16 + 1: return launch_backward_rows<DT, WDT, 4, 1>(a, st);
  case 8 * 16 + 1: return launch_backward_rows<DT, WDT, 8, 1>(a, st);
  case 16 * 16 + 1: return launch_backward_rows<DT, WDT, 16, 1>(a, st);
  case 32 * 16 + 1: return launch_backward_rows<DT, WDT, 32, 1>(a, st);
  case 64 * 16 + 1: return launch_backward_rows<DT, WDT, 64, 1>(a, st);
  case 64 * 16 + 2: return launch_backward_rows<DT, WDT, 64, 2>(a, st);
  case 64 * 16 + 3: return launch_backward_rows<DT, WDT, 64, 3>(a, st);
  case 64 * 16 + 4: return launch_backward_rows<DT, WDT, 64, 4>(a, st);
  case 128 * 16 + 3: return launch_backward_rows<DT, WDT, 128, 3>(a, st);
  case 128 * 16 + 4: return launch_backward_rows<DT, WDT, 128, 4>(a, st);
  case 256 * 16 + 3: return launch_backward_rows<DT, WDT, 256, 3>(a, st);
  case 256 * 16 + 4: return launch_backward_rows<DT, WDT, 256, 4>(a, st);
  case 1024 * 16 + 2: return launch_backward_rows<DT, WDT, 1024, 2>(a, st);
  }
  if (a.rows > 0) {
    hipError_t e = launch_statistics<DT, WDT, true>(a, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ln_columns_kernel<DT, WDT>), dim3((unsigned)(a.cols / (kLNThreads * V)), (unsigned)a.nparts),
                       dim3(kLNThreads), 0, st, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return launch_reduce<WDT, kLNThreads, V>(a, st);
}

} // namespace sb

hipError_t sb_launch_layer_norm(const sb::LNArgs &a, int dtype, int wdtype, hipStream_t st) {
  using namespace sb;
  if (dtype == DT_F32) return launch_forward<DT_F32, DT_F32>(a, st);
  if (dtype == DT_F16)
    return wdtype == DT_F32 ? launch_forward<DT_F16, DT_F32>(a, st) : launch_forward<DT_F16, DT_F16>(a, st);
  return wdtype == DT_F32 ? launch_forward<DT_BF16, DT_F32>(a, st) : launch_forward<DT_BF16, DT_BF16>(a, st);
}

hipError_t sb_launch_layer_norm_backward(const sb::LNArgs &a, int dtype, int wdtype, hipStream_t st) {
  using namespace sb;
  if (dtype == DT_F32) return launch_backward<DT_F32, DT_F32>(a, st);
  if (dtype == DT_F16)
    return wdtype == DT_F32 ? launch_backward<DT_F16, DT_F32>(a, st) : launch_backward<DT_F16, DT_F16>(a, st);
  return wdtype == DT_F32 ? launch_backward<DT_BF16, DT_F32>(a, st) : launch_backward<DT_BF16, DT_BF16>(a, st);
}
