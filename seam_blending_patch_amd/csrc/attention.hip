// attention.hip -- attention forward for gfx950: softmax(scale q k^T) v with the
// scores kept in registers, and the joining of splits over the keys.
#include "attention_tile.h"

namespace sb {
namespace {

// Forward.  A wave has 32 rows (query, head of the group), a lane one of them:
// S^T = K Q^T puts a row's scores into one lane and its partner in the other
// half, so a row's maximum and sum need one exchange, a row's factors are
// scalars of a lane, and P^T feeds O^T += V^T P^T as it lies.
template <int DT, int DP, int NW>
__global__ __launch_bounds__(64 * NW) void attention_kernel(const AttnArgs a) {
  constexpr int kThreads = 64 * NW;
  constexpr int KT = NW > 1 && Tile<DT, DP, 32>::SC <= 16 ? 64 : 32, NS = KT / 32; // keys of a tile
  using T = Tile<DT, DP, KT>;
  using St = Stage<DT, DP, KT, kThreads>;
  constexpr bool kAhead = St::N <= 8;     // the next tile is requested while this one is used
  constexpr int kBufs = kAhead ? 2 : 1, NB = DP / 32, PW = DT == DT_F32 ? 16 : 8;
  __shared__ alignas(16) char lds[kBufs][2][T::kBytes];

  const Work w = work_of(a);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5, n = lane & 31;
  const int klen = length_of(a.k_len, w.b, a.Lk), qlen = length_of(a.q_len, w.b, a.Lq);
  const int off = klen - qlen, live_rows = qlen * a.group;
  const int r0 = w.tile * 32 * NW, wr0 = r0 + wave * 32, row = wr0 + n;
  const bool live = row < live_rows;
  // keys that a row sees: the first seen(row)
  const auto seen = [&](int r) {
    return a.causal ? min(max((int)fdiv((uint32_t)r, a.div_group) + off + 1, 0), klen) : klen;
  };
  const int sees = live ? seen(row) : klen;          // (rows past the end compute something that is not kept)
  const int sure = seen(min(wr0, max(live_rows - 1, 0))); // keys that all rows of the wave see
  const int last = min(r0 + 32 * NW, live_rows) - 1, wlast = min(wr0 + 32, live_rows) - 1;
  const int begin = w.split * a.span;
  const int end = last < r0 ? 0 : min(seen(last), begin + a.span);
  const int wend = wlast < wr0 ? 0 : min(seen(wlast), end);

  u32x4 qf[T::kFrags];
  {
    const int64_t at = live ? row_at(a.q, a, w.b, w.hk, row) : 0;
#pragma unroll
    for (int u = 0; u < T::kFrags; ++u) qf[u] = load_chunk<DT>(a.q.p, at, 2 * u + h, a.D, live);
  }
  f32x16 o[NB];
#pragma unroll
  for (int db = 0; db < NB; ++db) o[db] = f32x16{0};
  float m = -kInf, l = 0.0f; // m: of the scores before scaling; l: of this lane's half of the keys
  const float slack = 8.0f / a.scale2;

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
      float s[NS][16];
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        f32x16 c = {0};
#pragma unroll
        for (int u = 0; u < T::kFrags; ++u) c = mma<DT>(T::row_fragment(kt, 32 * j + n, u, h), qf[u], c);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[j][i] = c[i];
      }
      if (k0 + KT > sure) {
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            s[j][i] = k0 + 32 * j + 8 * (i >> 2) + 4 * h + (i & 3) < sees ? s[j][i] : -kInf;
      }
      float mx = s[0][0];
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[j][i]);
      mx = half_max(mx);
      // The running maximum only has to keep exp2 in range: it moves when some
      // row's has grown by 2^8 or more (P is then at most 2^8, which 16 bits
      // hold as exactly as 1), which spares most tiles the turn over O.
      if (__any(mx > m + slack)) {
        const float up = fmaxf(m, mx), by = m == -kInf ? 0.0f : __builtin_amdgcn_exp2f((m - up) * a.scale2);
        m = up;
        l *= by;
#pragma unroll
        for (int db = 0; db < NB; ++db) o[db] = o[db] * by;
      }
      const float base = m == -kInf ? 0.0f : -m * a.scale2;
      uint32_t p[NS][PW];
#pragma unroll
      for (int j = 0; j < NS; ++j) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[j][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][i], a.scale2, base));
          l += s[j][i];
        }
        pack_operand<DT>(s[j], p[j]);
      }
#pragma unroll
      for (int db = 0; db < NB; ++db)
#pragma unroll
        for (int j = 0; j < NS; ++j) o[db] = T::column_product(vt, 32 * j, db, p[j], o[db], lane);
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
  l = half_sum(l);
  const bool some = live && !(l == 0.0f); // (a NaN goes on)
  const float by = some ? 1.0f / l : 0.0f;
  const float lse = some ? m * a.scale + logf(l) : -kInf;
  if (a.part_lse) {
    const int64_t at = ((int64_t)w.split * a.B * a.Hk + w.unit) * a.rows + row;
    if (h == 0) a.part_lse[at] = lse;
#pragma unroll
    for (int db = 0; db < NB; ++db)
      store_column<DT_F32>(a.part, at * a.D, db, h, a.D, some ? o[db] : f32x16{0}, by);
  } else {
    if (a.lse && h == 0) a.lse[stat_at(a, w.b, w.hk, row)] = lse;
    const int64_t at = row_at(a.out, a, w.b, w.hk, row);
#pragma unroll
    for (int db = 0; db < NB; ++db)
      store_column<DT>((void *)a.out.p, at, db, h, a.D, some ? o[db] : f32x16{0}, by);
  }
}

// A wave joins the splits of a row: out = sum_s exp(lse_s - lse) out_s.  At most
// 64 splits: a lane has the weight of one.
constexpr int kJoinRows = 4; // rows of a block
template <int DT> __global__ __launch_bounds__(64 * kJoinRows) void join_kernel(const AttnArgs a, int64_t count) {
  const int lane = threadIdx.x & 63;
  const int64_t at = (int64_t)blockIdx.x * kJoinRows + (threadIdx.x >> 6);
  if (at >= count) return;
  const float lse = lane < a.splits ? a.part_lse[lane * count + at] : -kInf;
  float most = lse;
#pragma unroll
  for (int k = 32; k; k >>= 1) most = fmaxf(most, __shfl_xor(most, k));
  const float weight = lse == -kInf ? 0.0f : __builtin_amdgcn_exp2f((lse - most) * kLog2e);
  const float total = lanes_sum<64>(weight);
  const bool some = !(total == 0.0f);
  const float mine = some ? weight / total : 0.0f;
  f32x4v acc = {0, 0, 0, 0};
  const int d = lane * 4, n = a.D - d;
  for (int s = 0; s < a.splits; ++s) {
    const float by = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), s));
    if (by == 0.0f || n <= 0) continue;
    const Vec<16> v = load_part<DT_F32>(a.part, (s * count + at) * a.D + d, n);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += by * __uint_as_float(v.w[i]);
  }
  const uint32_t unit = (uint32_t)(at / a.rows);
  const int row = (int)(at - (int64_t)unit * a.rows), b = (int)fdiv(unit, a.div_Hk), hk = (int)(unit - b * a.div_Hk.d);
  if (a.lse && lane == 0) a.lse[stat_at(a, b, hk, row)] = some ? most + logf(total) : -kInf;
  const int64_t to = row_at(a.out, a, b, hk, row);
  store_four<DT>((void *)a.out.p, to + d, n, acc);
}

// A gradient's splits added up in their order: rows [units][len][D] of the
// partial results to head hk * group + g of sample b, position r / group
template <int DT>
__global__ __launch_bounds__(64 * kJoinRows) void sum_kernel(const AttnHeads out, const float *part, int splits, int D,
                                                             int64_t count, int64_t len, FastDiv div_group,
                                                             FastDiv div_Hk) {
  const int lane = threadIdx.x & 63;
  const int64_t at = (int64_t)blockIdx.x * kJoinRows + (threadIdx.x >> 6);
  if (at >= count) return;
  const int d = lane * 4, n = D - d;
  f32x4v acc = {0, 0, 0, 0};
  for (int s = 0; s < splits; ++s) {
    const Vec<16> v = load_part<DT_F32>(part, (s * count + at) * D + d, n);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += __uint_as_float(v.w[i]);
  }
  const uint32_t unit = (uint32_t)(at / len), r = (uint32_t)(at - (int64_t)unit * len);
  const uint32_t b = fdiv(unit, div_Hk), hk = unit - b * div_Hk.d, q = fdiv(r, div_group), g = r - q * div_group.d;
  store_four<DT>((void *)out.p, b * out.b + q * out.t + (int64_t)(hk * div_group.d + g) * out.h + d, n, acc);
}

template <int DT, int DP> void launch(const AttnArgs &a, int waves, hipStream_t st) {
  if (waves == 1) hipLaunchKernelGGL((attention_kernel<DT, DP, 1>), dim3(a.blocks), dim3(64), 0, st, a);
  else
    hipLaunchKernelGGL((attention_kernel<DT, DP, kAttnWaves>), dim3(a.blocks), dim3(64 * kAttnWaves), 0, st, a);
}
template <int DT> hipError_t launch(const AttnArgs &a, int waves, hipStream_t st) {
  switch (attn_padded(a.D)) {
  case 32: launch<DT, 32>(a, waves, st); break;
  case 64: launch<DT, 64>(a, waves, st); break;
  case 96: launch<DT, 96>(a, waves, st); break;
  case 128: launch<DT, 128>(a, waves, st); break;
  case 160: launch<DT, 160>(a, waves, st); break;
  case 192: launch<DT, 192>(a, waves, st); break;
  default: launch<DT, 256>(a, waves, st);
  }
  return hipGetLastError();
}

} // namespace
} // namespace sb

hipError_t sb_launch_attention(const sb::AttnArgs &a, int dtype, int waves, hipStream_t st) {
  if (dtype == sb::DT_F32) return sb::launch<sb::DT_F32>(a, waves, st);
  if (dtype == sb::DT_F16) return sb::launch<sb::DT_F16>(a, waves, st);
  return sb::launch<sb::DT_BF16>(a, waves, st);
}

hipError_t sb_launch_attention_join(const sb::AttnArgs &a, int dtype, hipStream_t st) {
  const int64_t count = (int64_t)a.B * a.Hk * a.rows;
  const dim3 grid((unsigned)((count + sb::kJoinRows - 1) / sb::kJoinRows)), block(64 * sb::kJoinRows);
  if (dtype == sb::DT_F32) hipLaunchKernelGGL((sb::join_kernel<sb::DT_F32>), grid, block, 0, st, a, count);
  else if (dtype == sb::DT_F16) hipLaunchKernelGGL((sb::join_kernel<sb::DT_F16>), grid, block, 0, st, a, count);
  else hipLaunchKernelGGL((sb::join_kernel<sb::DT_BF16>), grid, block, 0, st, a, count);
  return hipGetLastError();
}

hipError_t sb_launch_attention_sum(const sb::AttnArgs &a, const sb::AttnHeads &out, const float *part, int64_t len,
                                   int group, int dtype, hipStream_t st) {
  const int64_t count = (int64_t)a.B * a.Hk * len;
  const dim3 grid((unsigned)((count + sb::kJoinRows - 1) / sb::kJoinRows)), block(64 * sb::kJoinRows);
  const sb::FastDiv dg = sb::make_fastdiv((uint32_t)group);
#define SB_SUM(DT) \
  hipLaunchKernelGGL((sb::sum_kernel<DT>), grid, block, 0, st, out, part, a.splits, a.D, count, len, dg, a.div_Hk)
  if (dtype == sb::DT_F32) SB_SUM(sb::DT_F32);
  else if (dtype == sb::DT_F16) SB_SUM(sb::DT_F16);
  else SB_SUM(sb::DT_BF16);
#undef SB_SUM
  return hipGetLastError();
}
