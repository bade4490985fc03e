// attention_backward.hip -- attention's gradients for gfx950.  The probabilities
// are formed again from the scores and their rows' log sums:
//   P = exp(scale q k^T - lse), delta = row sums of dout * out,
//   dS = P (dout v^T - delta), dq = scale dS k, dk = scale dS^T q, dv = P^T dout.
// Two kernels, one for dq (and delta) that goes along the keys, one for dk and dv
// that goes along the rows: each result has one owner that adds it up in a fixed
// order, at the price of forming S and dout v^T twice (7 products for 5, in 16 bits 8:
// Left below).
//
// Roundings to 16 bits: P and dS where they enter a product (the matrix cores' rate in
// 16 bits is 8 times that in fp32).  That of out, which delta is formed of, is taken out
// again.  Errors of dq and dk against 64 bits, relative, 10140 tokens of heads of 128
// bf16: 2.2e-3 and 2.4e-3, 1.7e-3 for the results' own rounding alone (3.5e-3 with out's
// rounding left in); fp16 an eighth.  fp32 rounds nothing.
#include "attention_tile.h"

namespace sb {
namespace {

// fp16 reaches from 6e-8 (6e-5 at full precision) to 65504 only, so what is packed into
// it is lifted by powers of two that the results are divided by again: P by 2^14, and dS
// by 2^4 over the norm of its row's dout (dk's kernel: the largest of its rows), rounded
// up to a power of two, less where out's norm passes 2^8.  |dS| <= P |dout| (|v| + |out|),
// so nothing passes fp16's range while values have norms up to 2000, however dout is
// scaled; and dS keeps full precision down to 4e-6 of dout's norm.  (dout of 1e-3 over
// 4096 keys of heads of 128, emulated: dq's error 2.8e-4, 9e-4 without.)  The loops have as
// many instructions with it: lifts are part of the log sums, and of a multiply-add in place
// of a subtraction (1537, 769 and 0 causal tokens 110 -> 112 us).
template <int DT> constexpr bool kLifts = DT == DT_F16;
template <int DT> constexpr int kLiftP = kLifts<DT> ? 14 : 0;
constexpr int kLiftS = 4;
struct Lift {
  float by, undo; // of dp - delta beside P's, of dS
  // the square of dout's norm, larger where out's norm is large
  static __device__ __forceinline__ float size(float dout_square, float out_square) {
    return dout_square * fmaxf(1.0f, out_square * 0x1p-16f);
  }
  // the power of two, at most 33 in size, that the norm is rounded up to (0 for infinity and NaN)
  static __device__ __forceinline__ int power(float square) { return (__builtin_amdgcn_frexp_expf(square) + 1) >> 1; }
  template <int DT> static __device__ __forceinline__ Lift of(int power) {
    if constexpr (!kLifts<DT>) return Lift{1.0f, 1.0f};
    return Lift{__int_as_float((127 + kLiftS - kLiftP<DT> - power) << 23), __int_as_float((127 + power - kLiftS) << 23)};
  }
};
// P (dp - delta): of P as lifted, and delta times `by`
template <int DT> __device__ __forceinline__ float gradient_of(float p, float dp, float delta, float by) {
  if constexpr (kLifts<DT>) return p * __builtin_fmaf(dp, by, -delta);
  else return p * (dp - delta);
}
// the largest size of a wave's 32 rows, for dk's kernel (an infinite one would say nothing
// of the others, and leaves nothing to lift in what it reaches)
__device__ __forceinline__ void store_peak(const AttnArgs &a, const Work &w, int row0, int lane, float square) {
  square = square < kInf ? square : 0.0f;
#pragma unroll
  for (int k = 16; k; k >>= 1) square = fmaxf(square, __shfl_xor(square, k));
  if (lane == 0 && w.split == 0 && row0 < a.rows) a.peak[(int64_t)w.unit * ((a.rows + 31) / 32) + row0 / 32] = square;
}
// and the power of that of rows begin (a multiple of 32) to end - 1 (none: 0), for a block
__device__ __forceinline__ int read_peak(const AttnArgs &a, const Work &w, int begin, int end, float *lds) {
  const float *const peak = a.peak + (int64_t)w.unit * ((a.rows + 31) / 32);
  const int blocks = (end + 31) / 32;
  float most = 0.0f;
  for (int i0 = begin / 32 + (int)threadIdx.x; i0 < blocks; i0 += 4 * 64 * kAttnWaves) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = peak[min(i0 + j * 64 * kAttnWaves, blocks - 1)];
#pragma unroll
    for (int j = 0; j < 4; ++j) most = fmaxf(most, v[j]);
  }
#pragma unroll
  for (int k = 32; k; k >>= 1) most = fmaxf(most, __shfl_xor(most, k));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = most;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAttnWaves; ++i) most = fmaxf(most, lds[i]);
  return __builtin_amdgcn_readfirstlane(Lift::power(most)); // (the same in every lane)
}

// What a row of dq still needs when its keys are done, in 16 bits (fp32: out's rounding
// is one of fp32, nothing is left).  delta is formed of an `out` that was rounded, and
// each dS was: with r = the sum of the row's dS, which is zero but for these,
//   dq = scale (sum dS k - r m),  m = sum P k,
// takes both out along m, and delta + the sum of dS before its rounding is the exact
// delta that dk's kernel needs.  The price is a product more, of the fragments that dS
// takes, and as many registers for m as for dq: 10140 tokens of 12 heads of 128 bf16 dq
// 1.38 ms, 0.93 without (when two columns of 32 rows to a wave had room); 8192 of 16 heads of
// 64 0.61 and 0.54; a pass of its own for delta would form two products again.
template <int DT> constexpr bool kMeanOf = DT != DT_F32;
template <int DT> struct Left {
  float rounded, exact;
  __device__ __forceinline__ void add(float ds) { exact += ds; }
  __device__ __forceinline__ void add(uint32_t packed) { rounded = pair_sum<DT>(packed, rounded); }
};

// A row's results: dq (columns from 32 db0 on), or the split's share of it with what
// is left, and delta.
template <int DT, int NB, int NM>
__device__ __forceinline__ void store_dq(const AttnArgs &a, const Work &w, int row, int h, int db0, bool live, float delta,
                                         float undo, Left<DT> left, f32x16 (&dq)[NB], const f32x16 (&mean)[NM]) {
  constexpr float kUnlift = 1.0f / (1 << kLiftP<DT>);
  if constexpr (kMeanOf<DT>) {
    left.rounded = half_sum(left.rounded);
    left.exact = half_sum(left.exact) * undo;
  }
  if (row >= a.rows) return;
  const float by = live ? a.scale * undo : 0.0f;
  const bool first = h == 0 && db0 == 0;
  if (a.part) {
    const int64_t at = ((int64_t)w.split * a.B * a.Hk + w.unit) * a.rows + row;
#pragma unroll
    for (int db = 0; db < NB; ++db)
      store_column<DT_F32>(a.part, at * a.D, db0 + db, h, a.D, live ? dq[db] : f32x16{0}, by);
    if constexpr (kMeanOf<DT>) {
#pragma unroll
      for (int db = 0; db < NB; ++db)
        store_column<DT_F32>(a.part_mean, at * a.D, db0 + db, h, a.D, live ? mean[db] : f32x16{0}, a.scale * kUnlift);
      if (first) {
        float *const to = a.part_left + 2 * at;
        to[0] = live ? left.rounded * undo : 0.0f;
        to[1] = live ? left.exact : 0.0f;
      }
    }
    if (live && first && w.split == 0) a.delta[stat_at(a, w.b, w.hk, row)] = delta;
  } else {
    const int64_t at = row_at(a.dq, a, w.b, w.hk, row);
    left.rounded *= kUnlift;
#pragma unroll
    for (int db = 0; db < NB; ++db) {
      if constexpr (kMeanOf<DT>) {
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[db][i] = __builtin_fmaf(-left.rounded, mean[db][i], dq[db][i]);
      }
      store_column<DT>((void *)a.dq.p, at, db0 + db, h, a.D, live ? dq[db] : f32x16{0}, by);
    }
    if (live && first) a.delta[stat_at(a, w.b, w.hk, row)] = kMeanOf<DT> ? delta + left.exact : delta;
  }
}

// dq.  As forward: a lane has a row; S^T = K Q^T, (dout v^T)^T = V dOut^T, and
// dS^T feeds dQ^T += K^T dS^T.  PAIR: a head is too long for one wave's registers; two
// waves have half of its elements of the same rows each, and add up their halves of
// the scores, of dout v^T and of delta through LDS.
template <int DT, int DP, int NW, bool PAIR>
__global__ __launch_bounds__(64 * NW) void dq_kernel(const AttnArgs a) {
  constexpr int kThreads = 64 * NW, KT = 32, W = PAIR ? 2 : 1, ROWS = 32 * NW / W;
  using T = Tile<DT, DP, KT>;
  using St = Stage<DT, DP, KT, kThreads>;
  constexpr int NF = T::kFrags / W, NB = DP / 32 / W, PW = DT == DT_F32 ? 16 : 8;
  constexpr bool kAhead = St::N <= 8 && NF * 4 <= 64; // the next tile is requested while this one is used
  constexpr int kBufs = kAhead ? 2 : 1;
  constexpr bool kMean = kMeanOf<DT>;
  __shared__ alignas(1024) char lds[kBufs * 2 * T::kBytes]; // of each buffer keys, then values
  __shared__ float halves[PAIR ? NW : 1][PAIR ? 32 : 1][64];

  const Work w = work_of<true>(a);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5, n = lane & 31;
  const int part = PAIR ? wave & 1 : 0;
  const int klen = length_of(a.k_len, w.b, a.Lk), qlen = length_of(a.q_len, w.b, a.Lq);
  const int off = klen - qlen, live_rows = qlen * a.group;
  const int r0 = w.tile * ROWS, wr0 = r0 + wave / W * 32, row = wr0 + n;
  const bool live = row < live_rows;
  const auto seen = [&](int r) {
    return a.causal ? min(max((int)fdiv((uint32_t)r, a.div_group) + off + 1, 0), klen) : klen;
  };
  const int sees = live ? seen(row) : klen;
  const int sure = seen(min(wr0, max(live_rows - 1, 0)));
  const int last = min(r0 + ROWS, live_rows) - 1, wlast = min(wr0 + 32, live_rows) - 1;
  const int begin = w.split * a.span;
  const int end = last < r0 ? 0 : min(seen(last), begin + a.span);
  const int wend = wlast < wr0 ? 0 : min(seen(wlast), end);

  u32x4 qf[NF], gf[NF];
  float delta = 0.0f, square = 0.0f, out_square = 0.0f, lse2 = kInf; // (a row that sees no key, or is none: its probabilities are exp2(-inf))
  Left<DT> left = {};
  {
    const int64_t at = live ? row_at(a.q, a, w.b, w.hk, row) : 0, to = live ? row_at(a.out, a, w.b, w.hk, row) : 0,
                  gt = live ? row_at(a.dout, a, w.b, w.hk, row) : 0;
#pragma unroll
    for (int u = 0; u < NF; ++u) {
      const int c = 2 * (u + part * NF) + h;
      qf[u] = load_chunk<DT>(a.q.p, at, c, a.D, live);
      gf[u] = load_chunk<DT>(a.dout.p, gt, c, a.D, live);
      const u32x4 of = load_chunk<DT>(a.out.p, to, c, a.D, live);
      float f[T::V], g[T::V];
      unpack<DT, 16>(Vec<16>{of[0], of[1], of[2], of[3]}, f);
      unpack<DT, 16>(Vec<16>{gf[u][0], gf[u][1], gf[u][2], gf[u][3]}, g);
#pragma unroll
      for (int i = 0; i < T::V; ++i) {
        delta = __builtin_fmaf(f[i], g[i], delta);
        if constexpr (kLifts<DT>) {
          square = __builtin_fmaf(g[i], g[i], square);
          out_square = __builtin_fmaf(f[i], f[i], out_square);
        }
      }
    }
    delta = half_sum(delta);
    if constexpr (kLifts<DT>) {
      square = half_sum(square);
      out_square = half_sum(out_square);
    }
    if constexpr (PAIR) {
      halves[wave][0][lane] = delta;
      halves[wave][1][lane] = square;
      halves[wave][2][lane] = out_square;
      __syncthreads();
      delta += halves[wave ^ 1][0][lane];
      square += halves[wave ^ 1][1][lane];
      out_square += halves[wave ^ 1][2][lane];
      __syncthreads();
    }
    if constexpr (kLifts<DT>) {
      square = Lift::size(square, out_square);
      if (part == 0) store_peak(a, w, wr0, lane, square);
    }
    if (live) {
      const int64_t st = stat_at(a, w.b, w.hk, row);
      const float lse = a.lse[st];
      if (lse != -kInf) lse2 = lse * kLog2e - kLiftP<DT>;
    }
  }
  const Lift lift = Lift::of<DT>(Lift::power(square));
  const float lifted = delta * lift.by;
  f32x16 dq[NB], mean[kMean ? NB : 1];
#pragma unroll
  for (int db = 0; db < NB; ++db) dq[db] = f32x16{0};
#pragma unroll
  for (int db = 0; db < (kMean ? NB : 1); ++db) mean[db] = f32x16{0};

  const int64_t k_base = w.b * a.k.b + w.hk * a.k.h, v_base = w.b * a.v.b + w.hk * a.v.h;
  const auto k_at = [&](int r) { return k_base + r * a.k.t; };
  const auto v_at = [&](int r) { return v_base + r * a.v.t; };
  const int row_lane = T::row_place(lane), col_lane = T::column_place(lane);
  St sk, sv;
  if (kAhead && begin < end) {
    sk.load(a.k.p, begin, klen, a.D, k_at);
    sv.load(a.v.p, begin, klen, a.D, v_at);
    sk.store(lds);
    sv.store(lds + T::kBytes);
    __syncthreads();
  }
  for (int k0 = begin, cur = 0; k0 < end; k0 += KT) {
    if constexpr (kAhead) {
      if (k0 + KT < end) {
        sk.load(a.k.p, k0 + KT, klen, a.D, k_at);
        sv.load(a.v.p, k0 + KT, klen, a.D, v_at);
      }
    } else {
      __syncthreads();
      stage_tile<DT, DP, KT, kThreads>(lds, a.k.p, k0, klen, a.D, k_at);
      stage_tile<DT, DP, KT, kThreads>(lds + T::kBytes, a.v.p, k0, klen, a.D, v_at);
      __syncthreads();
    }
    const int kt = row_lane + cur, vt = kt + T::kBytes, kc = col_lane + cur;
    if (PAIR || k0 < wend) {
      f32x16 s = {0}, dp = {0};
#pragma unroll
      for (int u = 0; u < NF; ++u) {
        s = mma<DT>(T::row_fragment(lds, kt, 0, u + part * NF), qf[u], s);
        dp = mma<DT>(T::row_fragment(lds, vt, 0, u + part * NF), gf[u], dp);
      }
      if constexpr (PAIR) { // (the barrier before the next tile keeps these until they are read)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          halves[wave][i][lane] = s[i];
          halves[wave][16 + i][lane] = dp[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[i] += halves[wave ^ 1][i][lane];
          dp[i] += halves[wave ^ 1][16 + i][lane];
        }
      }
      float p[16], ds[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], a.scale2, -lse2));
        ds[i] = gradient_of<DT>(p[i], dp[i], lifted, lift.by);
      }
      if (k0 + KT > sure) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool sees_it = k0 + 8 * (i >> 2) + 4 * h + (i & 3) < sees;
          p[i] = sees_it ? p[i] : 0.0f;
          ds[i] = sees_it ? ds[i] : 0.0f;
        }
      }
      uint32_t pp[PW], pd[PW];
      pack_operand<DT>(ds, pd);
      if constexpr (kMean) {
        pack_operand<DT>(p, pp);
#pragma unroll
        for (int i = 0; i < 16; ++i) left.add(ds[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) left.add(pd[i]);
      }
#pragma unroll
      for (int db = 0; db < NB; ++db) {
        dq[db] = T::column_product(lds, kc, 0, db + part * NB, pd, dq[db]);
        if constexpr (kMean) mean[db] = T::column_product(lds, kc, 0, db + part * NB, pp, mean[db]);
      }
    }
    if constexpr (kAhead) {
      cur ^= 2 * T::kBytes;
      if (k0 + KT < end) {
        sk.store(lds + cur);
        sv.store(lds + cur + T::kBytes);
      }
      __syncthreads();
    }
  }

  store_dq<DT, NB>(a, w, row, h, part * NB, live, delta, lift.undo, left, dq, mean);
}

// dk and dv.  A lane has a key: S = Q K^T and dOut V^T put the rows into its
// registers, and P and dS feed dV^T += dOut^T P and dK^T += Q^T dS.  K and V stay
// in registers, rows come through LDS.  PAIR: a head is too long for one wave's
// registers; two waves have half of its elements each, and add up their halves of
// S and dOut V^T through LDS.
template <int DT, int DP, bool PAIR>
__global__ __launch_bounds__(64 * kAttnWaves) void dkv_kernel(const AttnArgs a) {
  constexpr int kThreads = 64 * kAttnWaves, RT = 32, KEYS = 32 * kAttnWaves / (PAIR ? 2 : 1);
  using T = Tile<DT, DP, RT>;
  using St = Stage<DT, DP, RT, kThreads>;
  constexpr int kBufs = 4 * T::kBytes <= 65536 * (PAIR ? 1 : 2) ? 2 : 1;
  constexpr bool kAhead = kBufs == 2;
  constexpr int W = PAIR ? 2 : 1, NF = T::kFrags / W, NB = DP / 32 / W, PW = DT == DT_F32 ? 16 : 8;
  __shared__ alignas(1024) char lds[kBufs * 2 * T::kBytes]; // of each buffer q, then dout
  __shared__ alignas(16) float stats[kBufs][2][RT]; // log sums (base 2) and deltas
  __shared__ float halves[PAIR ? kAttnWaves : 1][PAIR ? 32 : 1][64];
  __shared__ float peaks[kAttnWaves];

  const Work w = work_of<false>(a);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5, n = lane & 31;
  const int part = PAIR ? wave & 1 : 0;
  const int klen = length_of(a.k_len, w.b, a.Lk), qlen = length_of(a.q_len, w.b, a.Lq);
  const int off = klen - qlen, live_rows = qlen * a.group;
  const int k0 = w.tile * KEYS, wk0 = k0 + (wave / W) * 32, key = wk0 + n;
  const bool live = key < klen;
  // rows that see a key: from first(key) on
  const auto first = [&](int k) { return a.causal ? max(k - off, 0) * a.group : 0; };
  const int from = first(key), wfrom = first(wk0), wsure = first(wk0 + 31);
  const int begin = max(w.split * a.span, first(k0) / RT * RT);
  const int end = k0 >= klen ? 0 : min(live_rows, w.split * a.span + a.span);

  u32x4 kf[NF], vf[NF];
#pragma unroll
  for (int u = 0; u < NF; ++u) {
    const int c = 2 * (u + part * NF) + h;
    kf[u] = load_chunk<DT>(a.k.p, w.b * a.k.b + w.hk * a.k.h + (live ? key : 0) * a.k.t, c, a.D, live);
    vf[u] = load_chunk<DT>(a.v.p, w.b * a.v.b + w.hk * a.v.h + (live ? key : 0) * a.v.t, c, a.D, live);
  }
  f32x16 dk[NB], dv[NB];
#pragma unroll
  for (int db = 0; db < NB; ++db) dk[db] = dv[db] = f32x16{0};

  const auto q_at = [&](int r) { return row_at(a.q, a, w.b, w.hk, r); };
  const auto g_at = [&](int r) { return row_at(a.dout, a, w.b, w.hk, r); };
  const int row_lane = T::row_place(lane), col_lane = T::column_place(lane);
  St sq, sg;
  Lift lift = Lift::of<DT>(0);
  if constexpr (kLifts<DT>) lift = Lift::of<DT>(read_peak(a, w, begin, end, peaks));
  float stat[2];
  const auto load_stats = [&](int r) { // of row r + thread
    stat[0] = kInf;                    // (no row: no probability)
    stat[1] = 0.0f;
    const int at = r + (int)threadIdx.x;
    if (threadIdx.x < RT && at < live_rows) {
      const int64_t st = stat_at(a, w.b, w.hk, at);
      const float lse = a.lse[st];
      if (lse != -kInf) stat[0] = lse * kLog2e - kLiftP<DT>;
      stat[1] = a.delta[st] * lift.by;
    }
  };
  const auto store_stats = [&](int buf) {
    if (threadIdx.x < RT) {
      stats[buf][0][threadIdx.x] = stat[0];
      stats[buf][1][threadIdx.x] = stat[1];
    }
  };
  if (kAhead && begin < end) {
    sq.load(a.q.p, begin, live_rows, a.D, q_at);
    sg.load(a.dout.p, begin, live_rows, a.D, g_at);
    load_stats(begin);
    sq.store(lds);
    sg.store(lds + T::kBytes);
    store_stats(0);
    __syncthreads();
  }
  for (int r0 = begin, cur = 0; r0 < end; r0 += RT) {
    if constexpr (kAhead) {
      if (r0 + RT < end) {
        sq.load(a.q.p, r0 + RT, live_rows, a.D, q_at);
        sg.load(a.dout.p, r0 + RT, live_rows, a.D, g_at);
        load_stats(r0 + RT);
      }
    } else {
      __syncthreads();
      load_stats(r0);
      stage_tile<DT, DP, RT, kThreads>(lds, a.q.p, r0, live_rows, a.D, q_at);
      stage_tile<DT, DP, RT, kThreads>(lds + T::kBytes, a.dout.p, r0, live_rows, a.D, g_at);
      store_stats(0);
      __syncthreads();
    }
    const int qt = row_lane + cur, gt = qt + T::kBytes, qc = col_lane + cur, gc = qc + T::kBytes;
    if (PAIR || r0 + RT > wfrom) {
      f32x16 s = {0}, dp = {0};
#pragma unroll
      for (int u = 0; u < NF; ++u) {
        s = mma<DT>(T::row_fragment(lds, qt, 0, u + part * NF), kf[u], s);
        dp = mma<DT>(T::row_fragment(lds, gt, 0, u + part * NF), vf[u], dp);
      }
      if constexpr (PAIR) { // (the barrier before the next tile keeps these until they are read)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          halves[wave][i][lane] = s[i];
          halves[wave][16 + i][lane] = dp[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[i] += halves[wave ^ 1][i][lane];
          dp[i] += halves[wave ^ 1][16 + i][lane];
        }
      }
      float p[16], ds[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 lse2 = *reinterpret_cast<const float4 *>(&stats[cur != 0][0][8 * j + 4 * h]);
        const float4 delta = *reinterpret_cast<const float4 *>(&stats[cur != 0][1][8 * j + 4 * h]);
        const float l4[4] = {lse2.x, lse2.y, lse2.z, lse2.w}, d4[4] = {delta.x, delta.y, delta.z, delta.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[4 * j + i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[4 * j + i], a.scale2, -l4[i]));
          ds[4 * j + i] = gradient_of<DT>(p[4 * j + i], dp[4 * j + i], d4[i], lift.by);
        }
      }
      if (r0 < wsure) { // causal: some row of the tile does not see some key of the wave
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool sees = r0 + 8 * (i >> 2) + 4 * h + (i & 3) >= from;
          p[i] = sees ? p[i] : 0.0f;
          ds[i] = sees ? ds[i] : 0.0f;
        }
      }
      uint32_t pp[PW], pd[PW];
      pack_operand<DT>(p, pp);
      pack_operand<DT>(ds, pd);
#pragma unroll
      for (int db = 0; db < NB; ++db) {
        dv[db] = T::column_product(lds, gc, 0, db + part * NB, pp, dv[db]);
        dk[db] = T::column_product(lds, qc, 0, db + part * NB, pd, dk[db]);
      }
    }
    if constexpr (kAhead) {
      cur ^= 2 * T::kBytes;
      if (r0 + RT < end) {
        sq.store(lds + cur);
        sg.store(lds + cur + T::kBytes);
        store_stats(cur != 0);
      }
      __syncthreads();
    }
  }

  if (key >= a.Lk) return;
  const float by = live ? a.scale * lift.undo : 0.0f;
  constexpr float kUnlift = 1.0f / (1 << kLiftP<DT>);
  const int64_t units = (int64_t)a.B * a.Hk, at = ((int64_t)w.split * units + w.unit) * a.Lk + key;
#pragma unroll
  for (int db = 0; db < NB; ++db) {
    const f32x16 k = live ? dk[db] : f32x16{0}, v = live ? dv[db] : f32x16{0};
    const int d = db + part * NB;
    if (a.part) {
      store_column<DT_F32>(a.part, at * a.D, d, h, a.D, k, by);
      store_column<DT_F32>(a.part, ((int64_t)a.splits * units * a.Lk + at) * a.D, d, h, a.D, v, kUnlift);
    } else {
      store_column<DT>((void *)a.dk.p, w.b * a.dk.b + w.hk * a.dk.h + key * a.dk.t, d, h, a.D, k, by);
      store_column<DT>((void *)a.dv.p, w.b * a.dv.b + w.hk * a.dv.h + key * a.dv.t, d, h, a.D, v, kUnlift);
    }
  }
}

// ---------------------------------------------------------------------------
// The same two gradients for 16-bit heads of up to 192, of whole chunks: every turn
// multiplies the next tile's scores while it turns this tile's into probabilities,
// an element beside each product, so that one wave keeps the matrix cores and the
// vector unit at work together.  Three buffers: the turn of tile t reads tiles t and
// t + 1 and stores tile t + 2.  Straight through, without a branch around products:
// with one the compiler carries the sums from one kind of register to the other and
// back (dk and dv 2.71 ms with the branches that spare a wave tiles it does not see,
// 1.86 without).  10140 tokens of 12 heads of 128 bf16: dq 1.38 ms (910 TFLOP/s on its four
// products), dk and dv 1.41 ms (900); 8192 tokens of 16 heads of 64 0.61 and 0.62 ms.
// Reading 12 products ahead in place of 6 loses (heads of 64 1.61 ms against 1.22 in all,
// with three products for dq).
// ---------------------------------------------------------------------------
constexpr int kProductsAhead = 6; // LDS reads this many products before their use

// Waits for all that was requested, in every lane: threads that store no chunk would
// leave it open to the compiler whether they still wait for theirs, and it would wait
// again between the next requests (dq of 10140 tokens of 12 heads of 128 bf16: 1.43 ms, 1.77
// without this).
__device__ __forceinline__ void arrived() { __builtin_amdgcn_s_waitcnt(0x0F70); } // (vmcnt 0, no other counter)

// dq: a wave has 32 rows.  (Two columns of them to a wave, where there are registers for
// that: 8192 tokens of 16 heads of 64 bf16 1229 us in all, so 1208.)
template <int DT, int DP> __global__ __launch_bounds__(64 * kAttnWaves) void dq_pipelined_kernel(const AttnArgs a) {
  constexpr int kThreads = 64 * kAttnWaves, KT = 32;
  using T = Tile<DT, DP, KT>;
  using St = RowStage<DT, DP, KT, kThreads>;
  constexpr int NB = DP / 32, NF = T::kFrags;
  __shared__ alignas(1024) char lds[3 * 2 * T::kBytes]; // of each buffer keys, then values

  const Work w = work_of<true>(a);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5, n = lane & 31;
  const int klen = length_of(a.k_len, w.b, a.Lk), qlen = length_of(a.q_len, w.b, a.Lq);
  const int off = klen - qlen, live_rows = qlen * a.group;
  const int r0 = w.tile * 32 * kAttnWaves, wr0 = r0 + wave * 32, row = wr0 + n;
  const bool live = row < live_rows;
  const auto seen = [&](int r) {
    return a.causal ? min(max((int)fdiv((uint32_t)r, a.div_group) + off + 1, 0), klen) : klen;
  };
  const int sees = live ? seen(row) : klen;
  const int sure = seen(min(wr0, max(live_rows - 1, 0)));
  const int last = min(r0 + 32 * kAttnWaves, live_rows) - 1;
  const int begin = w.split * a.span;
  const int end = last < r0 ? 0 : min(seen(last), begin + a.span);

  u32x4 qf[NF], gf[NF];
  float delta = 0.0f, square = 0.0f, out_square = 0.0f, lse2 = kInf; // (lse2: as in dq_kernel)
  {
    const int64_t at = live ? row_at(a.q, a, w.b, w.hk, row) : 0, to = live ? row_at(a.out, a, w.b, w.hk, row) : 0,
                  gt = live ? row_at(a.dout, a, w.b, w.hk, row) : 0;
#pragma unroll
    for (int u = 0; u < NF; ++u) {
      qf[u] = load_chunk<DT>(a.q.p, at, 2 * u + h, a.D, live);
      gf[u] = load_chunk<DT>(a.dout.p, gt, 2 * u + h, a.D, live);
      const u32x4 of = load_chunk<DT>(a.out.p, to, 2 * u + h, a.D, live);
      float f[T::V], g[T::V];
      unpack<DT, 16>(Vec<16>{of[0], of[1], of[2], of[3]}, f);
      unpack<DT, 16>(Vec<16>{gf[u][0], gf[u][1], gf[u][2], gf[u][3]}, g);
#pragma unroll
      for (int i = 0; i < T::V; ++i) {
        delta = __builtin_fmaf(f[i], g[i], delta);
        if constexpr (kLifts<DT>) {
          square = __builtin_fmaf(g[i], g[i], square);
          out_square = __builtin_fmaf(f[i], f[i], out_square);
        }
      }
    }
    delta = half_sum(delta);
    if constexpr (kLifts<DT>) {
      square = Lift::size(half_sum(square), half_sum(out_square));
      store_peak(a, w, wr0, lane, square);
    }
    if (live) {
      const float lse = a.lse[stat_at(a, w.b, w.hk, row)];
      if (lse != -kInf) lse2 = lse * kLog2e - kLiftP<DT>;
    }
  }
  const Lift lift = Lift::of<DT>(Lift::power(square));
  const float lifted = delta * lift.by;
  f32x16 dq[NB], mean[NB];
  Left<DT> left = {};
#pragma unroll
  for (int db = 0; db < NB; ++db) dq[db] = mean[db] = f32x16{0};

  const int row_lane = T::row_place(lane), col_lane = T::column_place(lane);
  const int tiles = end > begin ? (end - begin + KT - 1) / KT : 0;
  if (tiles) {
    clear_tiles<kThreads>(lds, sizeof lds, a.D < DP);
    St sk, sv;
    sk.start(a.k.p, w.b * a.k.b + w.hk * a.k.h, a.k.t, begin, a.D);
    sv.start(a.v.p, w.b * a.v.b + w.hk * a.v.h, a.v.t, begin, a.D);
    sk.load(begin, klen);
    sv.load(begin, klen);
    sk.store(lds);
    sv.store(lds + T::kBytes);
    if (tiles > 1) {
      sk.load(begin + KT, klen);
      sv.load(begin + KT, klen);
      sk.store(lds + 2 * T::kBytes);
      sv.store(lds + 3 * T::kBytes);
    }
    if (tiles > 2) {
      sk.load(begin + 2 * KT, klen);
      sv.load(begin + 2 * KT, klen);
    }
    __syncthreads();
    f32x16 s = {0}, dp = {0}, s1, dp1;
    // steps: for each fragment u the keys' and the values'
    const auto read = [&](int buffer, int i) {
      return T::row_fragment(lds, row_lane + buffer + (i & 1) * T::kBytes, 0, i >> 1);
    };
    in_order<2 * NF, kProductsAhead>([&](int i) { return read(0, i); }, [&](int i, u32x4 f) {
      if (i & 1) dp = mma<DT>(f, gf[i >> 1], dp);
      else s = mma<DT>(f, qf[i >> 1], s);
    });
    int b0 = 0, b1 = 2 * T::kBytes, b2 = 4 * T::kBytes;
    for (int t = 0, k0 = begin; t < tiles; ++t, k0 += KT) {
      if (t + 2 < tiles) {
        arrived();
        sk.store(lds + b2);
        sv.store(lds + b2 + T::kBytes);
        if (t + 3 < tiles) {
          sk.load(k0 + 3 * KT, klen);
          sv.load(k0 + 3 * KT, klen);
        }
      }
      {
        float p[16], ds[16];
        s1 = dp1 = f32x16{0};
        // (behind the last tile: scores of what the buffer holds, not used)
        uint32_t pp[8], pd[8];
        in_order<2 * NF + 2 * NB, kProductsAhead>(
            [&](int i) {
              const int j = i - 2 * NF;
              return j < 0 ? read(b1, i) : T::column_fragment(lds, col_lane + b0, 0, j % NB, j / NB);
            },
            [&](int i, u32x4 f) {
              const int j = i - 2 * NF;
              if (j >= 0) {
                const uint32_t *q = pd + 4 * (j / NB), *m = pp + 4 * (j / NB);
                dq[j % NB] = mma<DT>(f, u32x4{q[0], q[1], q[2], q[3]}, dq[j % NB]);
                mean[j % NB] = mma<DT>(f, u32x4{m[0], m[1], m[2], m[3]}, mean[j % NB]);
                // (beside the products: the sums, and the second half's packing)
#pragma unroll
                for (int e = j * 8 / NB; e < (j + 1) * 8 / NB; ++e) left.add(ds[e]);
                if (j == NB - 1) {
#pragma unroll
                  for (int e = 4; e < 8; ++e) {
                    pp[e] = pack_pair<DT>(p + 2 * e);
                    pd[e] = pack_pair<DT>(ds + 2 * e);
                  }
                }
#pragma unroll
                for (int e = j * 4 / NB; e < (j + 1) * 4 / NB; ++e) left.add(pd[e]);
                return;
              }
              if (i & 1) dp1 = mma<DT>(f, gf[i >> 1], dp1);
              else s1 = mma<DT>(f, qf[i >> 1], s1);
#pragma unroll
              for (int e = i * 16 / (2 * NF); e < (i + 1) * 16 / (2 * NF); ++e) {
                p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], a.scale2, -lse2));
                ds[e] = gradient_of<DT>(p[e], dp[e], lifted, lift.by);
              }
              if (j == -1) {
                if (k0 + KT > sure) {
                  const int keys = sees - k0 - 4 * h;
#pragma unroll
                  for (int x = 0; x < 16; ++x) {
                    p[x] = 8 * (x >> 2) + (x & 3) < keys ? p[x] : 0.0f;
                    ds[x] = 8 * (x >> 2) + (x & 3) < keys ? ds[x] : 0.0f;
                  }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  pp[e] = pack_pair<DT>(p + 2 * e);
                  pd[e] = pack_pair<DT>(ds + 2 * e);
                }
              }
            });
        s = s1;
        dp = dp1;
      }
      lds_barrier();
      const int b = b0;
      b0 = b1;
      b1 = b2;
      b2 = b;
    }
  }

  store_dq<DT, NB>(a, w, row, h, 0, live, delta, lift.undo, left, dq, mean);
}

// dk and dv: a wave has 32 keys.
template <int DT, int DP> __global__ __launch_bounds__(64 * kAttnWaves) void dkv_pipelined_kernel(const AttnArgs a) {
  constexpr int kThreads = 64 * kAttnWaves, RT = 32, KEYS = 32 * kAttnWaves;
  using T = Tile<DT, DP, RT>;
  using S = Share<DT, DP, RT, kThreads>;
  constexpr int NF = T::kFrags, NB = DP / 32;
  __shared__ alignas(1024) char lds[3 * 2 * T::kBytes]; // of each buffer q, then dout
  __shared__ alignas(16) float stats[3][2][RT];         // log sums (base 2) and deltas
  __shared__ float peaks[kAttnWaves];

  const Work w = work_of<false>(a);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5, n = lane & 31;
  const int klen = length_of(a.k_len, w.b, a.Lk), qlen = length_of(a.q_len, w.b, a.Lq);
  const int off = klen - qlen, live_rows = qlen * a.group;
  const int k0 = w.tile * KEYS, wk0 = k0 + wave * 32, key = wk0 + n;
  const bool live = key < klen;
  // rows that see a key: from first(key) on
  const auto first = [&](int k) { return a.causal ? max(k - off, 0) * a.group : 0; };
  const int from = first(key), wsure = first(wk0 + 31);
  const int begin = max(w.split * a.span, first(k0) / RT * RT);
  const int end = k0 >= klen ? 0 : min(live_rows, w.split * a.span + a.span);

  u32x4 kf[NF], vf[NF];
#pragma unroll
  for (int u = 0; u < NF; ++u) {
    kf[u] = load_chunk<DT>(a.k.p, w.b * a.k.b + w.hk * a.k.h + (live ? key : 0) * a.k.t, 2 * u + h, a.D, live);
    vf[u] = load_chunk<DT>(a.v.p, w.b * a.v.b + w.hk * a.v.h + (live ? key : 0) * a.v.t, 2 * u + h, a.D, live);
  }
  f32x16 dk[NB], dv[NB];
#pragma unroll
  for (int db = 0; db < NB; ++db) dk[db] = dv[db] = f32x16{0};

  Lift lift = Lift::of<DT>(0);
  if constexpr (kLifts<DT>) lift = Lift::of<DT>(read_peak(a, w, begin, end, peaks));
  u32x4 sq[S::N], sg[S::N];
  float stat[2];
  const bool any = S::chunk() * T::V < a.D && !(S::kIdle && S::row(0) >= RT);
  const int e0 = any ? S::chunk() * T::V : 0;
  // A tile's packed rows are the last one's moved on where whole queries fill it:
  // then offsets are added to, not formed.
  const bool regular = RT % a.group == 0;
  const int64_t q_step = RT / a.group * a.q.t, g_step = RT / a.group * a.dout.t;
  int64_t q_off[S::N], g_off[S::N], st_off;
  const auto place = [&](int r) { // (rows past the end: the last one, whose probabilities are zeros then)
#pragma unroll
    for (int k = 0; k < S::N; ++k) {
      const int x = min(r + S::row(k), live_rows - 1);
      q_off[k] = row_at(a.q, a, w.b, w.hk, x) + e0;
      g_off[k] = row_at(a.dout, a, w.b, w.hk, x) + e0;
    }
    st_off = stat_at(a, w.b, w.hk, min(r + (int)threadIdx.x % RT, live_rows - 1));
  };
  const auto load = [&](int r) { // the tile of rows r on, the one after the last loaded
    typedef typename El<DT>::bits bits;
    if (!regular || r + RT > live_rows) place(r);
#pragma unroll
    for (int k = 0; k < S::N; ++k) {
      sq[k] = *reinterpret_cast<const typename El<DT>::vec *>((const bits *)a.q.p + q_off[k]);
      sg[k] = *reinterpret_cast<const typename El<DT>::vec *>((const bits *)a.dout.p + g_off[k]);
      q_off[k] += q_step;
      g_off[k] += g_step;
    }
    stat[0] = a.lse[st_off]; // (looked at when it is stored, so that nothing waits for it here)
    stat[1] = a.delta[st_off];
    st_off += RT / a.group;
  };
  const auto store = [&](int buffer, int r) {
    char *to = lds + buffer * 2 * T::kBytes;
    if (any) {
#pragma unroll
      for (int k = 0; k < S::N; ++k) {
        *reinterpret_cast<u32x4 *>(to + T::place(S::row(k), S::chunk())) = sq[k];
        *reinterpret_cast<u32x4 *>(to + T::kBytes + T::place(S::row(k), S::chunk())) = sg[k];
      }
    }
    if (threadIdx.x < RT) {
      // (no row, or one without keys: no probability)
      stats[buffer][0][threadIdx.x] = r + (int)threadIdx.x >= live_rows || stat[0] == -kInf ? kInf : stat[0] * kLog2e - kLiftP<DT>;
      stats[buffer][1][threadIdx.x] = stat[1] * lift.by;
    }
  };
  const int row_lane = T::row_place(lane), col_lane = T::column_place(lane);
  const int tiles = end > begin ? (end - begin + RT - 1) / RT : 0;
  if (tiles) {
    clear_tiles<kThreads>(lds, sizeof lds, a.D < DP);
    place(begin);
    load(begin);
    store(0, begin);
    if (tiles > 1) {
      load(begin + RT);
      store(1, begin + RT);
    }
    if (tiles > 2) load(begin + 2 * RT);
    __syncthreads();
    f32x16 s, dp, s1, dp1;
    const auto read = [&](int buffer, int i) { // the rows' q and dout by turns
      return T::row_fragment(lds, row_lane + buffer * 2 * T::kBytes + (i & 1) * T::kBytes, 0, i >> 1);
    };
    s = dp = f32x16{0};
    in_order<2 * NF, kProductsAhead>([&](int i) { return read(0, i); }, [&](int i, u32x4 f) {
      if (i & 1) dp = mma<DT>(f, vf[i >> 1], dp);
      else s = mma<DT>(f, kf[i >> 1], s);
    });
    int b0 = 0, b1 = 1, b2 = 2;
    for (int t = 0, r0 = begin; t < tiles; ++t, r0 += RT) {
      if (t + 2 < tiles) {
        store(b2, r0 + 2 * RT);
        if (t + 3 < tiles) load(r0 + 3 * RT);
      }
      {
        float p[16], ds[16];
        f32x4v lse2[4], delta[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          lse2[j] = *reinterpret_cast<const f32x4v *>(&stats[b0][0][8 * j + 4 * h]);
          delta[j] = *reinterpret_cast<const f32x4v *>(&stats[b0][1][8 * j + 4 * h]);
        }
        s1 = dp1 = f32x16{0};
        // (behind the last tile: scores of what the buffer holds, not used)
        uint32_t pp[8], pd[8];
        in_order<2 * NF + 4 * NB, kProductsAhead>(
            [&](int i) {
              const int j = i - 2 * NF;
              return j < 0 ? read(b1, i)
                           : T::column_fragment(lds, col_lane + b0 * 2 * T::kBytes + (j < 2 * NB ? T::kBytes : 0), 0, j % NB,
                                                j / NB % 2);
            },
            [&](int i, u32x4 f) {
              const int j = i - 2 * NF;
              if (j >= 0) {
                const uint32_t *q = (j < 2 * NB ? pp : pd) + 4 * (j / NB % 2);
                const u32x4 b = {q[0], q[1], q[2], q[3]};
                if (j < 2 * NB) dv[j % NB] = mma<DT>(f, b, dv[j % NB]);
                else dk[j % NB] = mma<DT>(f, b, dk[j % NB]);
                return;
              }
              if (i & 1) dp1 = mma<DT>(f, vf[i >> 1], dp1);
              else s1 = mma<DT>(f, kf[i >> 1], s1);
#pragma unroll
              for (int e = i * 16 / (2 * NF); e < (i + 1) * 16 / (2 * NF); ++e) {
                p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], a.scale2, -lse2[e >> 2][e & 3]));
                ds[e] = gradient_of<DT>(p[e], dp[e], delta[e >> 2][e & 3], lift.by);
              }
              if (j == -1) {
                if (r0 < wsure) { // causal: some row of the tile does not see some key of the wave
#pragma unroll
                  for (int x = 0; x < 16; ++x) {
                    const bool sees = r0 + 8 * (x >> 2) + 4 * h + (x & 3) >= from;
                    p[x] = sees ? p[x] : 0.0f;
                    ds[x] = sees ? ds[x] : 0.0f;
                  }
                }
                pack_operand<DT>(p, pp);
                pack_operand<DT>(ds, pd);
              }
            });
        s = s1;
        dp = dp1;
      }
      lds_barrier();
      const int b = b0;
      b0 = b1;
      b1 = b2;
      b2 = b;
    }
  }

  if (key >= a.Lk) return;
  const float by = live ? a.scale * lift.undo : 0.0f;
  constexpr float kUnlift = 1.0f / (1 << kLiftP<DT>);
  const int64_t units = (int64_t)a.B * a.Hk, at = ((int64_t)w.split * units + w.unit) * a.Lk + key;
#pragma unroll
  for (int db = 0; db < NB; ++db) {
    const f32x16 k = live ? dk[db] : f32x16{0}, v = live ? dv[db] : f32x16{0};
    if (a.part) {
      store_column<DT_F32>(a.part, at * a.D, db, h, a.D, k, by);
      store_column<DT_F32>(a.part, ((int64_t)a.splits * units * a.Lk + at) * a.D, db, h, a.D, v, kUnlift);
    } else {
      store_column<DT>((void *)a.dk.p, w.b * a.dk.b + w.hk * a.dk.h + key * a.dk.t, db, h, a.D, k, by);
      store_column<DT>((void *)a.dv.p, w.b * a.dv.b + w.hk * a.dv.h + key * a.dv.t, db, h, a.D, v, kUnlift);
    }
  }
}

// whole: heads of whole 16-byte chunks, which some kernels want
template <int DT, int DP> void launch_dq(const AttnArgs &a, int waves, int whole, hipStream_t st) {
  const dim3 grid(a.blocks), block(64 * kAttnWaves);
  if constexpr (attn_pipelined(Elem<DT>::bytes, DP)) {
    if (whole && waves > 1) {
      hipLaunchKernelGGL((dq_pipelined_kernel<DT, DP>), grid, block, 0, st, a);
      return;
    }
  }
  constexpr bool kPair = attn_dq_paired(Elem<DT>::bytes, DP);
  constexpr int kFew = kPair ? 2 : 1; // waves of a block of 32 rows
  if (waves == 1) hipLaunchKernelGGL((dq_kernel<DT, DP, kFew, kPair>), grid, dim3(64 * kFew), 0, st, a);
  else hipLaunchKernelGGL((dq_kernel<DT, DP, kAttnWaves, kPair>), grid, block, 0, st, a);
}
template <int DT, int DP> void launch_dkv(const AttnArgs &a, int whole, hipStream_t st) {
  const dim3 grid(a.blocks), block(64 * kAttnWaves);
  if constexpr (attn_pipelined(Elem<DT>::bytes, DP)) {
    if (whole) {
      hipLaunchKernelGGL((dkv_pipelined_kernel<DT, DP>), grid, block, 0, st, a);
      return;
    }
  }
  hipLaunchKernelGGL((dkv_kernel<DT, DP, attn_paired(Elem<DT>::bytes, DP)>), grid, block, 0, st, a);
}

// f(type, padded length) with both as constants
template <int DT, class F> void of_width(int padded, F f) {
  constexpr std::integral_constant<int, DT> dt{};
  switch (padded) {
  case 32: f(dt, std::integral_constant<int, 32>{}); break;
  case 64: f(dt, std::integral_constant<int, 64>{}); break;
  case 96: f(dt, std::integral_constant<int, 96>{}); break;
  case 128: f(dt, std::integral_constant<int, 128>{}); break;
  case 160: f(dt, std::integral_constant<int, 160>{}); break;
  case 192: f(dt, std::integral_constant<int, 192>{}); break;
  default: f(dt, std::integral_constant<int, 256>{});
  }
}
template <class F> hipError_t of_kind(int dtype, int D, F f) {
  if (dtype == DT_F32) of_width<DT_F32>(attn_padded(D), f);
  else if (dtype == DT_F16) of_width<DT_F16>(attn_padded(D), f);
  else of_width<DT_BF16>(attn_padded(D), f);
  return hipGetLastError();
}

} // namespace
} // namespace sb

hipError_t sb_launch_attention_dq(const sb::AttnArgs &a, int dtype, int waves, int whole, hipStream_t st) {
  return sb::of_kind(dtype, a.D, [&](auto dt, auto dp) { sb::launch_dq<dt(), dp()>(a, waves, whole, st); });
}
hipError_t sb_launch_attention_dkv(const sb::AttnArgs &a, int dtype, int whole, hipStream_t st) {
  return sb::of_kind(dtype, a.D, [&](auto dt, auto dp) { sb::launch_dkv<dt(), dp()>(a, whole, st); });
}
