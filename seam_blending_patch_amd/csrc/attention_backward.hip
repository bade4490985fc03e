// attention_backward.hip -- attention's gradients for gfx950.  The probabilities
// are formed again from the scores and their rows' log sums:
//   P = exp(scale q k^T - lse), delta = row sums of dout * out,
//   dS = P (dout v^T - delta), dq = scale dS k, dk = scale dS^T q, dv = P^T dout.
// Two kernels, one for dq (and delta) that goes along the keys, one for dk and dv
// that goes along the rows: each result has one owner that adds it up in a fixed
// order, at the price of forming S and dout v^T twice (7 products for 5).
#include "attention_tile.h"

namespace sb {
namespace {

// dq.  As forward: a lane has a row; S^T = K Q^T, (dout v^T)^T = V dOut^T, and
// dS^T feeds dQ^T += K^T dS^T.
template <int DT, int DP, int NW>
__global__ __launch_bounds__(64 * NW) void dq_kernel(const AttnArgs a) {
  constexpr int kThreads = 64 * NW, KT = 32;
  using T = Tile<DT, DP, KT>;
  using St = Stage<DT, DP, KT, kThreads>;
  constexpr bool kAhead = St::N <= 8 && T::kFrags * 4 <= 64; // the next tile is requested while this one is used
  constexpr int kBufs = kAhead ? 2 : 1, NB = DP / 32, PW = DT == DT_F32 ? 16 : 8;
  __shared__ alignas(16) char lds[kBufs][2][T::kBytes];

  const Work w = work_of(a);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5, n = lane & 31;
  const int klen = length_of(a.k_len, w.b, a.Lk), qlen = length_of(a.q_len, w.b, a.Lq);
  const int off = klen - qlen, live_rows = qlen * a.group;
  const int r0 = w.tile * 32 * NW, wr0 = r0 + wave * 32, row = wr0 + n;
  const bool live = row < live_rows;
  const auto seen = [&](int r) {
    return a.causal ? min(max((int)fdiv((uint32_t)r, a.div_group) + off + 1, 0), klen) : klen;
  };
  const int sees = live ? seen(row) : klen;
  const int sure = seen(min(wr0, max(live_rows - 1, 0)));
  const int last = min(r0 + 32 * NW, live_rows) - 1, wlast = min(wr0 + 32, live_rows) - 1;
  const int begin = w.split * a.span;
  const int end = last < r0 ? 0 : min(seen(last), begin + a.span);
  const int wend = wlast < wr0 ? 0 : min(seen(wlast), end);

  u32x4 qf[T::kFrags], gf[T::kFrags];
  float delta = 0.0f, lse2 = kInf; // (a row that sees no key, or is none: its probabilities are exp2(-inf))
  {
    const int64_t at = live ? row_at(a.q, a, w.b, w.hk, row) : 0, to = live ? row_at(a.out, a, w.b, w.hk, row) : 0,
                  gt = live ? row_at(a.dout, a, w.b, w.hk, row) : 0;
#pragma unroll
    for (int u = 0; u < T::kFrags; ++u) {
      qf[u] = load_chunk<DT>(a.q.p, at, 2 * u + h, a.D, live);
      gf[u] = load_chunk<DT>(a.dout.p, gt, 2 * u + h, a.D, live);
      const u32x4 of = load_chunk<DT>(a.out.p, to, 2 * u + h, a.D, live);
      float f[T::V], g[T::V];
      unpack<DT, 16>(Vec<16>{of[0], of[1], of[2], of[3]}, f);
      unpack<DT, 16>(Vec<16>{gf[u][0], gf[u][1], gf[u][2], gf[u][3]}, g);
#pragma unroll
      for (int i = 0; i < T::V; ++i) delta = __builtin_fmaf(f[i], g[i], delta);
    }
    delta = half_sum(delta);
    if (live) {
      const int64_t st = stat_at(a, w.b, w.hk, row);
      const float lse = a.lse[st];
      if (lse != -kInf) lse2 = lse * kLog2e;
      if (w.split == 0 && h == 0) a.delta[st] = delta;
    }
  }
  f32x16 dq[NB];
#pragma unroll
  for (int db = 0; db < NB; ++db) dq[db] = f32x16{0};

  const int64_t k_base = w.b * a.k.b + w.hk * a.k.h, v_base = w.b * a.v.b + w.hk * a.v.h;
  const auto k_at = [&](int r) { return k_base + r * a.k.t; };
  const auto v_at = [&](int r) { return v_base + r * a.v.t; };
  St sk, sv;
  if (kAhead && begin < end) {
    sk.load(a.k.p, begin, klen, a.D, k_at);
    sv.load(a.v.p, begin, klen, a.D, v_at);
    sk.store(lds[0][0]);
    sv.store(lds[0][1]);
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
      sk.load(a.k.p, k0, klen, a.D, k_at);
      sk.store(lds[0][0]);
      sv.load(a.v.p, k0, klen, a.D, v_at);
      sv.store(lds[0][1]);
      __syncthreads();
    }
    const char *kt = lds[cur][0], *vt = lds[cur][1];
    if (k0 < wend) {
      f32x16 s = {0}, dp = {0};
#pragma unroll
      for (int u = 0; u < T::kFrags; ++u) {
        s = mma<DT>(T::row_fragment(kt, n, u, h), qf[u], s);
        dp = mma<DT>(T::row_fragment(vt, n, u, h), gf[u], dp);
      }
      float ds[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        ds[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], a.scale2, -lse2)) * (dp[i] - delta);
      if (k0 + KT > sure) {
#pragma unroll
        for (int i = 0; i < 16; ++i) ds[i] = k0 + 8 * (i >> 2) + 4 * h + (i & 3) < sees ? ds[i] : 0.0f;
      }
      uint32_t p[PW];
      pack_operand<DT>(ds, p);
#pragma unroll
      for (int db = 0; db < NB; ++db) dq[db] = T::column_product(kt, 0, db, p, dq[db], lane);
    }
    if constexpr (kAhead) {
      cur ^= 1;
      if (k0 + KT < end) {
        sk.store(lds[cur][0]);
        sv.store(lds[cur][1]);
      }
      __syncthreads();
    }
  }

  if (row >= a.rows) return;
  const float by = live ? a.scale : 0.0f;
  if (a.part) {
    const int64_t at = ((int64_t)w.split * a.B * a.Hk + w.unit) * a.rows + row;
#pragma unroll
    for (int db = 0; db < NB; ++db)
      store_column<DT_F32>(a.part, at * a.D, db, h, a.D, live ? dq[db] : f32x16{0}, by);
  } else {
    const int64_t at = row_at(a.dq, a, w.b, w.hk, row);
#pragma unroll
    for (int db = 0; db < NB; ++db)
      store_column<DT>((void *)a.dq.p, at, db, h, a.D, live ? dq[db] : f32x16{0}, by);
  }
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
  __shared__ alignas(16) char lds[kBufs][2][T::kBytes];
  __shared__ alignas(16) float stats[kBufs][2][RT]; // log sums (base 2) and deltas
  __shared__ float halves[PAIR ? kAttnWaves : 1][PAIR ? 32 : 1][64];

  const Work w = work_of(a);
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
  St sq, sg;
  float stat[2];
  const auto load_stats = [&](int r) { // of row r + thread
    stat[0] = kInf;                    // (no row: no probability)
    stat[1] = 0.0f;
    const int at = r + (int)threadIdx.x;
    if (threadIdx.x < RT && at < live_rows) {
      const int64_t st = stat_at(a, w.b, w.hk, at);
      const float lse = a.lse[st];
      if (lse != -kInf) stat[0] = lse * kLog2e;
      stat[1] = a.delta[st];
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
    sq.store(lds[0][0]);
    sg.store(lds[0][1]);
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
      sq.load(a.q.p, r0, live_rows, a.D, q_at);
      sq.store(lds[0][0]);
      sg.load(a.dout.p, r0, live_rows, a.D, g_at);
      sg.store(lds[0][1]);
      store_stats(0);
      __syncthreads();
    }
    const char *qt = lds[cur][0], *gt = lds[cur][1];
    if (PAIR || r0 + RT > wfrom) {
      f32x16 s = {0}, dp = {0};
#pragma unroll
      for (int u = 0; u < NF; ++u) {
        s = mma<DT>(T::row_fragment(qt, n, u + part * NF, h), kf[u], s);
        dp = mma<DT>(T::row_fragment(gt, n, u + part * NF, h), vf[u], dp);
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
        const float4 lse2 = *reinterpret_cast<const float4 *>(&stats[cur][0][8 * j + 4 * h]);
        const float4 delta = *reinterpret_cast<const float4 *>(&stats[cur][1][8 * j + 4 * h]);
        const float l4[4] = {lse2.x, lse2.y, lse2.z, lse2.w}, d4[4] = {delta.x, delta.y, delta.z, delta.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[4 * j + i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[4 * j + i], a.scale2, -l4[i]));
          ds[4 * j + i] = p[4 * j + i] * (dp[4 * j + i] - d4[i]);
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
        dv[db] = T::column_product(gt, 0, db + part * NB, pp, dv[db], lane);
        dk[db] = T::column_product(qt, 0, db + part * NB, pd, dk[db], lane);
      }
    }
    if constexpr (kAhead) {
      cur ^= 1;
      if (r0 + RT < end) {
        sq.store(lds[cur][0]);
        sg.store(lds[cur][1]);
        store_stats(cur);
      }
      __syncthreads();
    }
  }

  if (key >= a.Lk) return;
  const float by = live ? a.scale : 0.0f;
  const int64_t units = (int64_t)a.B * a.Hk, at = ((int64_t)w.split * units + w.unit) * a.Lk + key;
#pragma unroll
  for (int db = 0; db < NB; ++db) {
    const f32x16 k = live ? dk[db] : f32x16{0}, v = live ? dv[db] : f32x16{0};
    const int d = db + part * NB;
    if (a.part) {
      store_column<DT_F32>(a.part, at * a.D, d, h, a.D, k, by);
      store_column<DT_F32>(a.part, ((int64_t)a.splits * units * a.Lk + at) * a.D, d, h, a.D, v, 1.0f);
    } else {
      store_column<DT>((void *)a.dk.p, w.b * a.dk.b + w.hk * a.dk.h + key * a.dk.t, d, h, a.D, k, by);
      store_column<DT>((void *)a.dv.p, w.b * a.dv.b + w.hk * a.dv.h + key * a.dv.t, d, h, a.D, v, 1.0f);
    }
  }
}

template <int DT, int DP> void launch_dq(const AttnArgs &a, int waves, hipStream_t st) {
  if (waves == 1) hipLaunchKernelGGL((dq_kernel<DT, DP, 1>), dim3(a.blocks), dim3(64), 0, st, a);
  else hipLaunchKernelGGL((dq_kernel<DT, DP, kAttnWaves>), dim3(a.blocks), dim3(64 * kAttnWaves), 0, st, a);
}
template <int DT, int DP> void launch_dkv(const AttnArgs &a, int, hipStream_t st) {
  hipLaunchKernelGGL((dkv_kernel<DT, DP, attn_paired(Elem<DT>::bytes, DP)>), dim3(a.blocks), dim3(64 * kAttnWaves), 0,
                     st, a);
}

#define SB_WIDTHS(F)                                                                                                   \
  template <int DT> hipError_t F(const AttnArgs &a, int waves, hipStream_t st) {                                      \
    switch (attn_padded(a.D)) {                                                                                        \
    case 32: F<DT, 32>(a, waves, st); break;                                                                           \
    case 64: F<DT, 64>(a, waves, st); break;                                                                           \
    case 96: F<DT, 96>(a, waves, st); break;                                                                           \
    case 128: F<DT, 128>(a, waves, st); break;                                                                         \
    case 160: F<DT, 160>(a, waves, st); break;                                                                         \
    case 192: F<DT, 192>(a, waves, st); break;                                                                         \
    default: F<DT, 256>(a, waves, st);                                                                                 \
    }                                                                                                                  \
    return hipGetLastError();                                                                                          \
  }                                                                                                                    \
  hipError_t F(const AttnArgs &a, int dtype, int waves, hipStream_t st) {                                              \
    if (dtype == DT_F32) return F<DT_F32>(a, waves, st);                                                               \
    if (dtype == DT_F16) return F<DT_F16>(a, waves, st);                                                               \
    return F<DT_BF16>(a, waves, st);                                                                                   \
  }
SB_WIDTHS(launch_dq)
SB_WIDTHS(launch_dkv)
#undef SB_WIDTHS

} // namespace
} // namespace sb

hipError_t sb_launch_attention_dq(const sb::AttnArgs &a, int dtype, int waves, hipStream_t st) {
  return sb::launch_dq(a, dtype, waves, st);
}
hipError_t sb_launch_attention_dkv(const sb::AttnArgs &a, int dtype, hipStream_t st) {
  return sb::launch_dkv(a, dtype, 0, st);
}
