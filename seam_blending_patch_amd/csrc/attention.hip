// attention.hip -- attention forward for gfx950: softmax(scale q k^T) v with the
// scores kept in registers, and the joining of splits over the keys.
#include "attention_tile.h"

namespace sb {
namespace {

// What a block of NW waves has to do, and a wave and a lane of it: a wave has 32
// rows (query, head of the group), a lane one of them.
template <int NW> struct Rows {
  Work w;
  int lane, h, row;        // row: of the unit, this lane's
  int klen, off, live_rows;
  int sees, sure;          // keys that the row sees: the first `sees`; that all rows of the wave see
  int begin, end, wend;    // keys of the block; the end of the wave's
  bool live;
  __device__ __forceinline__ int seen(const AttnArgs &a, int r) const {
    return a.causal ? min(max((int)fdiv((uint32_t)r, a.div_group) + off + 1, 0), klen) : klen;
  }
  __device__ __forceinline__ Rows(const AttnArgs &a) : w(work_of<true>(a)) {
    lane = threadIdx.x & 63;
    h = lane >> 5;
    klen = length_of(a.k_len, w.b, a.Lk);
    const int qlen = length_of(a.q_len, w.b, a.Lq), r0 = w.tile * 32 * NW, wr0 = r0 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 32;
    off = klen - qlen;
    live_rows = qlen * a.group;
    row = wr0 + (lane & 31);
    live = row < live_rows;
    sees = live ? seen(a, row) : klen; // (rows past the end compute something that is not kept)
    sure = seen(a, min(wr0, max(live_rows - 1, 0)));
    const int last = min(r0 + 32 * NW, live_rows) - 1, wlast = min(wr0 + 32, live_rows) - 1;
    begin = w.split * a.span;
    end = last < r0 ? 0 : min(seen(a, last), begin + a.span);
    wend = wlast < wr0 ? 0 : min(seen(a, wlast), end);
  }
};

// A wave's rows on their way: S^T = K Q^T puts a row's scores into one lane and
// its partner in the other half, so a row's maximum and sum need one exchange, a
// row's factors are scalars of a lane, and P^T feeds O^T += V^T P^T as it lies.
template <int DT, int DP, int KT> struct Softmax {
  using T = Tile<DT, DP, KT>;
  static constexpr int NS = KT / 32, NB = DP / 32, PW = DT == DT_F32 ? 16 : 8;
  // fp16: P and its sum are held times 2^7, up to 2^15, so that keys of 2^-32 of the
  // largest weight still count (one key of weight 1 and 30000 of 3e-8, whose values are
  // all the result, are lost without)
  static constexpr int kLift = DT == DT_F16 ? 7 : 0;
  u32x4 qf[T::kFrags];
  f32x16 o[NB];
  // P = exp2(s scale2 - c): c is near the row's largest exponent so far, less kLift, and is
  // exactly what the sums were formed with, so that moving them on to another c leaves
  // none of its rounding in the weights.  l: of this lane's half of the keys.
  float c, l;
  float s[NS][16];
  uint32_t p[NS][PW];

  template <int NW> __device__ __forceinline__ void start(const AttnArgs &a, const Rows<NW> &r) {
    const int64_t at = r.live ? row_at(a.q, a, r.w.b, r.w.hk, r.row) : 0;
#pragma unroll
    for (int u = 0; u < T::kFrags; ++u) qf[u] = load_chunk<DT>(a.q.p, at, 2 * u + r.h, a.D, r.live);
#pragma unroll
    for (int db = 0; db < NB; ++db) o[db] = f32x16{0};
    c = -kInf;
    l = 0.0f;
  }
  // Steps of the products: first those of P with the values (kMix of them), then
  // those of the keys with Q.
  static constexpr int kMix = DT == DT_F32 ? 0 : 2 * NS * NB, kScores = NS * T::kFrags, kAhead = 6;
  __device__ __forceinline__ u32x4 score_read(const char *lds, int kt, int i) const {
    return T::row_fragment(lds, kt, 32 * (i % NS), i / NS);
  }
  __device__ __forceinline__ void score_use(f32x16 (&c)[NS], int i, u32x4 f) const {
    c[i % NS] = mma<DT>(f, qf[i / NS], c[i % NS]);
  }
  __device__ __forceinline__ u32x4 mix_read(const char *lds, int vt, int i) const {
    return T::column_fragment(lds, vt, 32 * (i / NB / 2), i % NB, i / NB % 2);
  }
  __device__ __forceinline__ void mix_use(int i, u32x4 f) {
    const uint32_t *q = p[i / NB / 2] + 4 * (i / NB % 2);
    o[i % NB] = mma<DT>(f, u32x4{q[0], q[1], q[2], q[3]}, o[i % NB]);
  }
  // (left to the compiler's order: with several waves to a SIMD it is as good for heads
  // of 128 and better for 64, 8192 tokens of 16 heads 320 us against 367)
  // (all: D reaches the last 16 elements of the padded head, else their products are
  // left out: 2049 causal tokens of heads of 80 fp32 269 us, with them 286; 8192 tokens
  // of heads of 48 bf16 326 and 339)
  __device__ __forceinline__ void scores(const char *lds, int kt, bool all) {
    constexpr int kMost = T::kFrags - 8 / T::V;
    f32x16 c[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      c[j] = f32x16{0};
#pragma unroll
      for (int u = 0; u < kMost; ++u) c[j] = mma<DT>(T::row_fragment(lds, kt, 32 * j, u), qf[u], c[j]);
    }
    if (all) {
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int u = kMost; u < T::kFrags; ++u) c[j] = mma<DT>(T::row_fragment(lds, kt, 32 * j, u), qf[u], c[j]);
    }
    keep(c);
  }
  __device__ __forceinline__ void mix(const char *lds, int vt) {
#pragma unroll
    for (int db = 0; db < NB; ++db)
#pragma unroll
      for (int j = 0; j < NS; ++j) o[db] = T::column_product(lds, vt, 32 * j, db, p[j], o[db]);
  }
  // the values of one tile and the scores of the next, without a break
  __device__ __forceinline__ void mix_then_scores(const char *lds, int vt, int kt) {
    f32x16 c[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) c[j] = f32x16{0};
    in_order<kMix + kScores, kAhead>(
        [&](int i) { return i < kMix ? mix_read(lds, vt, i) : score_read(lds, kt, i - kMix); },
        [&](int i, u32x4 f) {
          if (i < kMix) mix_use(i, f);
          else score_use(c, i - kMix, f);
        });
    keep(c);
  }
  __device__ __forceinline__ void keep(const f32x16 (&c)[NS]) {
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[j][i] = c[j][i];
  }
  // left: how many of the tile's keys the row sees, less 4 h
  __device__ __forceinline__ void hide(int left) {
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[j][i] = 32 * j + 8 * (i >> 2) + (i & 3) < left ? s[j][i] : -kInf;
  }
  __device__ __forceinline__ void soften(float scale2) {
    float mx = s[0][0];
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[j][i]);
    mx = half_max(mx) * scale2 - kLift;
    // c only has to keep exp2 in range: it moves when some row's largest has grown by
    // 2^8 or more (P is at most 2^8 in between, which 16 bits hold as exactly as 1), which
    // spares most tiles the turn over O.  (fp16, exponents so large that their own
    // rounding counts in powers of two: that is what 2^8 are left to.)
    const float slack = kLift && !(fabsf(c) < 0x1p20f) ? 0.0f : 8.0f;
    if (__any(mx > c + slack)) {
      const float up = fmaxf(c, mx), by = c == -kInf ? 0.0f : __builtin_amdgcn_exp2f(c - up);
      c = up;
      l *= by;
#pragma unroll
      for (int db = 0; db < NB; ++db) o[db] = o[db] * by;
    }
    const float base = c == -kInf ? 0.0f : -c;
    // (a tile's own sum first: small weights behind a large one would be lost one by one)
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[j][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][i], scale2, base));
        sum += s[j][i];
      }
      pack_operand<DT>(s[j], p[j]);
    }
    l += sum;
  }
  template <int NW> __device__ __forceinline__ void finish(const AttnArgs &a, const Rows<NW> &r) {
    if (r.row >= a.rows) return;
    l = half_sum(l);
    const bool some = r.live && !(l == 0.0f); // (a NaN goes on)
    const float by = some ? 1.0f / l : 0.0f;
    const float lse = some ? __builtin_fmaf(c, kLn2, logf(l)) : -kInf;
    if (a.part_lse) {
      const int64_t at = ((int64_t)r.w.split * a.B * a.Hk + r.w.unit) * a.rows + r.row;
      if (r.h == 0) a.part_lse[at] = lse;
#pragma unroll
      for (int db = 0; db < NB; ++db)
        store_column<DT_F32>(a.part, at * a.D, db, r.h, a.D, some ? o[db] : f32x16{0}, by);
    } else {
      if (a.lse && r.h == 0) a.lse[stat_at(a, r.w.b, r.w.hk, r.row)] = lse;
      const int64_t at = row_at(a.out, a, r.w.b, r.w.hk, r.row);
#pragma unroll
      for (int db = 0; db < NB; ++db)
        store_column<DT>((void *)a.out.p, at, db, r.h, a.D, some ? o[db] : f32x16{0}, by);
    }
  }
};

// Blocks of one wave (single tokens: bound by memory, 4.3 TB/s over a cache of unlike
// lengths in the caches, 5.0 over one of 4096 keys each) or four, which take turns at the matrix
// cores as they come.  8192 tokens of 16 heads of 64 bf16: 320 us, 860 TFLOP/s, what
// the vector unit's work on the scores allows there; 2049 causal tokens of 16 heads
// of 80 fp32: 269 us, 80 TFLOP/s where a library product reaches 139 (a twelfth of it
// for the values' padding to 96, a third for the unequal tiles).
template <int DT, int DP, int NW>
__global__ __launch_bounds__(64 * NW, attn_forward_waves(Elem<DT>::bytes, DP, NW)) void attention_kernel(const AttnArgs a) {
  constexpr int kThreads = 64 * NW;
  constexpr int KT = NW > 1 && Tile<DT, DP, 32>::SC <= 16 ? 64 : 32; // keys of a tile
  using T = Tile<DT, DP, KT>;
  using St = Stage<DT, DP, KT, kThreads>;
  constexpr bool kAhead = St::N <= 8; // the next tile is requested while this one is used
  constexpr int kBufs = kAhead ? 2 : 1;
  __shared__ alignas(1024) char lds[kBufs * 2 * T::kBytes]; // of each buffer keys, then values

  const Rows<NW> r(a);
  Softmax<DT, DP, KT> x;
  x.start(a, r);
  const bool all = a.D > DP - 16;
  const int64_t k_base = r.w.b * a.k.b + r.w.hk * a.k.h, v_base = r.w.b * a.v.b + r.w.hk * a.v.h;
  const auto k_at = [&](int k) { return k_base + k * a.k.t; };
  const auto v_at = [&](int k) { return v_base + k * a.v.t; };
  const int row_lane = T::row_place(r.lane), col_lane = T::column_place(r.lane);
  St sk, sv;
  if (kAhead && r.begin < r.end) {
    sk.load(a.k.p, r.begin, r.klen, a.D, k_at);
    sv.load(a.v.p, r.begin, r.klen, a.D, v_at);
    sk.store(lds);
    sv.store(lds + T::kBytes);
    __syncthreads();
  }
  for (int k0 = r.begin, cur = 0; k0 < r.end; k0 += KT) {
    if constexpr (kAhead) {
      if (k0 + KT < r.end) {
        sk.load(a.k.p, k0 + KT, r.klen, a.D, k_at);
        sv.load(a.v.p, k0 + KT, r.klen, a.D, v_at);
      }
    } else {
      __syncthreads();
      stage_tile<DT, DP, KT, kThreads>(lds, a.k.p, k0, r.klen, a.D, k_at);
      stage_tile<DT, DP, KT, kThreads>(lds + T::kBytes, a.v.p, k0, r.klen, a.D, v_at);
      __syncthreads();
    }
    if (k0 < r.wend) {
      // (the wave that has products goes first, the other has a softmax to do meanwhile)
      __builtin_amdgcn_s_setprio(1);
      x.scores(lds, row_lane + cur, all);
      __builtin_amdgcn_s_setprio(0);
      if (k0 + KT > r.sure) x.hide(r.sees - k0 - 4 * r.h);
      x.soften(a.scale2);
      __builtin_amdgcn_s_setprio(1);
      x.mix(lds, col_lane + cur + T::kBytes);
      __builtin_amdgcn_s_setprio(0);
    }
    if constexpr (kAhead) {
      cur ^= 2 * T::kBytes;
      if (k0 + KT < r.end) {
        sk.store(lds + cur);
        sv.store(lds + cur + T::kBytes);
      }
      __syncthreads();
    }
  }
  x.finish(a, r);
}

// Many rows: blocks of 8 waves in two sets, one wave of each to a SIMD, half a
// turn apart: while one set has its products (of the last tile's values, of the
// next tile's keys) the other has its softmax, so the matrix cores and the vector
// unit are at work together instead of in turn.  Phases are kept apart by
// barriers; in phase 2 t (the second set: 2 t + 1) a wave multiplies tile t's keys,
// in the next it softens them, in the one after that it multiplies its values.
// Keys t + 2 and values t + 1 are stored while tile t is softened, in one of three
// buffers: its last reader was done two phases before, its first comes two after.
// 20280 tokens of 12 heads of 128 bf16: 2.65 ms, 940 TFLOP/s (2.8 ms in blocks of four
// waves; a library product reaches 1220).  The bound is LDS: a phase's fragments are
// 64 KiB by rows and 64 KiB by columns for four waves, at 115 and 82 bytes a clock
// 1370 clocks beside 1024 of products; without the softmax the rest takes 2.1 ms.
// Heads of 64 have half the products to a softmax and gain nothing (8192 tokens of 16
// 431 us against 320).
template <int DT, int DP>
__global__ __launch_bounds__(128 * kAttnWaves) void attention_wide_kernel(const AttnArgs a) {
  constexpr int NW = 2 * kAttnWaves, kThreads = 64 * NW;
  constexpr int KT = Tile<DT, DP, 32>::SC <= 16 ? 64 : 32; // keys of a tile
  using T = Tile<DT, DP, KT>;
  using St = RowStage<DT, DP, KT, kThreads>;
  __shared__ alignas(1024) char lds[3 * 2 * T::kBytes]; // of each buffer keys, then values

  const Rows<NW> r(a);
  Softmax<DT, DP, KT> x;
  x.start(a, r);
  const int64_t k_base = r.w.b * a.k.b + r.w.hk * a.k.h, v_base = r.w.b * a.v.b + r.w.hk * a.v.h;
  const int row_lane = T::row_place(r.lane), col_lane = T::column_place(r.lane);
  const int tiles = r.end > r.begin ? (r.end - r.begin + KT - 1) / KT : 0;
  if (tiles) {
    clear_tiles<kThreads>(lds, sizeof lds, a.D < DP);
    St sk, sv;
    sk.start(a.k.p, k_base, a.k.t, r.begin, a.D);
    sv.start(a.v.p, v_base, a.v.t, r.begin, a.D);
    sk.load(r.begin, r.klen);
    sv.load(r.begin, r.klen);
    sk.store(lds);
    sv.store(lds + T::kBytes);
    if (tiles > 1) {
      sk.load(r.begin + KT, r.klen);
      sv.load(r.begin + KT, r.klen);
      sk.store(lds + 2 * T::kBytes);
    }
    if (tiles > 2) sk.load(r.begin + 2 * KT, r.klen);
    __syncthreads();
    const bool second = __builtin_amdgcn_readfirstlane(threadIdx.x) >= kThreads / 2;
    if (second) lds_barrier();
    if (r.begin < r.wend) x.scores(lds, row_lane, true);
    // byte offsets of the buffers of tiles t, t + 1 and t + 2
    int b0 = 0, b1 = 2 * T::kBytes, b2 = 4 * T::kBytes;
    for (int t = 0, k0 = r.begin; t < tiles; ++t, k0 += KT) {
      lds_barrier();
      if (k0 < r.wend) {
        if (k0 + KT > r.sure) x.hide(r.sees - k0 - 4 * r.h);
        x.soften(a.scale2);
      }
      if (t + 2 < tiles) {
        sk.store(lds + b2);
        if (t + 3 < tiles) sk.load(k0 + 3 * KT, r.klen);
      }
      if (t + 1 < tiles) {
        sv.store(lds + b1 + T::kBytes);
        if (t + 2 < tiles) sv.load(k0 + 2 * KT, r.klen);
      }
      lds_barrier();
      // (behind the last tile the scores are those of what the buffer holds, and not used)
      if (k0 < r.wend) x.mix_then_scores(lds, col_lane + b0 + T::kBytes, row_lane + b1);
      const int b = b0;
      b0 = b1;
      b1 = b2;
      b2 = b;
    }
    if (!second) lds_barrier();
  }
  x.finish(a, r);
}

// Joins the splits of a row (8 tokens of 32 heads of 128 from 64 splits 5 us): out = sum_s exp(lse_s - lse) out_s.  At most 64
// splits: a lane has the weight of one.  WAVES waves to a row, each with some of
// the splits, 8 of which it requests together.
constexpr int kJoinRows = 4; // waves of a block
template <int DT, int WAVES> __global__ __launch_bounds__(64 * kJoinRows) void join_kernel(const AttnArgs a, int64_t count) {
  __shared__ f32x4v lds[kJoinRows][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, part = wave % WAVES;
  const int64_t at = (int64_t)blockIdx.x * (kJoinRows / WAVES) + wave / WAVES;
  const bool any = at < count;
  const float lse = any && lane < a.splits ? a.part_lse[lane * count + at] : -kInf;
  const int d = lane * 4, n = any ? a.D - d : 0;
  Vec<16> v[8]; // (the first are on their way while the weights are formed)
  const auto request = [&](int s0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int s = s0 + j * WAVES;
      v[j] = load_part<DT_F32>(a.part, (s * count + at) * a.D + d, s < a.splits ? n : 0);
    }
  };
  request(part);
  float most = lse;
#pragma unroll
  for (int k = 32; k; k >>= 1) most = fmaxf(most, __shfl_xor(most, k));
  const float weight = lse == -kInf ? 0.0f : __builtin_amdgcn_exp2f((lse - most) * kLog2e);
  const float total = lanes_sum<64>(weight);
  const bool some = !(total == 0.0f);
  const float mine = some ? weight / total : 0.0f;
  f32x4v acc = {0, 0, 0, 0};
  for (int s0 = part; s0 < a.splits; s0 += 8 * WAVES) {
    if (s0 != part) request(s0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float by = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), min(s0 + j * WAVES, 63)));
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(by, __uint_as_float(v[j].w[i]), acc[i]);
    }
  }
  if constexpr (WAVES > 1) {
    lds[wave][lane] = acc;
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int w = 1; w < WAVES; ++w) acc += lds[wave + w][lane];
  }
  if (!any) return;
  const uint32_t unit = (uint32_t)(at / a.rows);
  const int row = (int)(at - (int64_t)unit * a.rows), b = (int)fdiv(unit, a.div_Hk), hk = (int)(unit - b * a.div_Hk.d);
  if (a.lse && lane == 0) a.lse[stat_at(a, b, hk, row)] = some ? most + logf(total) : -kInf;
  const int64_t to = row_at(a.out, a, b, hk, row);
  store_four<DT>((void *)a.out.p, to + d, n, acc);
}

// Gradients' splits added up in their order: 4 elements to a thread.
struct SumArgs {
  AttnHeads out[2];
  const float *part;
  int splits, D;
  int64_t rows, len;      // of all units, of one
  FastDiv div_quads;      // 4-element steps of a row
  FastDiv div_group, div_Hk;
};
constexpr int kSumThreads = 256;
template <int DT> __global__ __launch_bounds__(kSumThreads) void sum_kernel(const SumArgs a) {
  const uint32_t row = blockIdx.x * (kSumThreads / a.div_quads.d) + fdiv(threadIdx.x, a.div_quads);
  const int d = (int)(threadIdx.x % a.div_quads.d) * 4, n = a.D - d;
  if (threadIdx.x >= kSumThreads / a.div_quads.d * a.div_quads.d || row >= a.rows) return;
  f32x4v acc = {0, 0, 0, 0};
  const float *part = a.part + (int64_t)blockIdx.y * a.splits * a.rows * a.D;
  for (int s0 = 0; s0 < a.splits; s0 += 8) {
    Vec<16> v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = load_part<DT_F32>(part, ((s0 + j) * a.rows + row) * a.D + d, s0 + j < a.splits ? n : 0);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += __uint_as_float(v[j].w[i]);
  }
  const uint32_t unit = (uint32_t)(row / a.len), r = (uint32_t)(row - (int64_t)unit * a.len);
  const uint32_t b = fdiv(unit, a.div_Hk), hk = unit - b * a.div_Hk.d, q = fdiv(r, a.div_group), g = r - q * a.div_group.d;
  const AttnHeads &out = a.out[blockIdx.y];
  store_four<DT>((void *)out.p, b * out.b + q * out.t + (int64_t)(hk * a.div_group.d + g) * out.h + d, n, acc);
}

// dq's splits added up the same way, less what their sums left of the row times its
// mean key; and delta with it (its row's first thread, behind its own splits' loads).
template <int DT> __global__ __launch_bounds__(kSumThreads) void dq_join_kernel(const AttnArgs a, const FastDiv div_quads,
                                                                                int64_t rows) {
  const uint32_t row = blockIdx.x * (kSumThreads / div_quads.d) + fdiv(threadIdx.x, div_quads);
  const int d = (int)(threadIdx.x % div_quads.d) * 4, n = a.D - d;
  if (threadIdx.x >= kSumThreads / div_quads.d * div_quads.d || row >= rows) return;
  f32x4v acc = {0, 0, 0, 0}, mean = {0, 0, 0, 0};
  float left = 0.0f, exact = 0.0f;
  for (int s0 = 0; s0 < a.splits; s0 += 8) {
    Vec<16> v[8], m[8];
    float2 l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool any = s0 + j < a.splits;
      const int64_t at = (any ? s0 + j : 0) * rows + row;
      v[j] = load_part<DT_F32>(a.part, at * a.D + d, any ? n : 0);
      m[j] = load_part<DT_F32>(a.part_mean, at * a.D + d, any ? n : 0);
      l[j] = *reinterpret_cast<const float2 *>(a.part_left + 2 * at);
      if (!any) l[j] = float2{0.0f, 0.0f};
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i] += __uint_as_float(v[j].w[i]);
        mean[i] += __uint_as_float(m[j].w[i]);
      }
      left += l[j].x;
      exact += l[j].y;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(-left, mean[i], acc[i]);
  const uint32_t unit = (uint32_t)(row / (uint32_t)a.rows), b = fdiv(unit, a.div_Hk), hk = unit - b * a.div_Hk.d;
  const int r = (int)(row - unit * (uint32_t)a.rows);
  store_four<DT>((void *)a.dq.p, row_at(a.dq, a, b, hk, r) + d, n, acc);
  if (d == 0 && r < length_of(a.q_len, b, a.Lq) * a.group) a.delta[stat_at(a, b, hk, r)] += exact;
}

template <int DT, int DP> void launch(const AttnArgs &a, int waves, hipStream_t st) {
  if (waves == 1) hipLaunchKernelGGL((attention_kernel<DT, DP, 1>), dim3(a.blocks), dim3(64), 0, st, a);
  else if (waves == kAttnWaves || !attn_wide(Elem<DT>::bytes, DP))
    hipLaunchKernelGGL((attention_kernel<DT, DP, kAttnWaves>), dim3(a.blocks), dim3(64 * kAttnWaves), 0, st, a);
  else if constexpr (attn_wide(Elem<DT>::bytes, DP))
    hipLaunchKernelGGL((attention_wide_kernel<DT, DP>), dim3(a.blocks), dim3(128 * kAttnWaves), 0, st, a);
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
  const int waves = a.splits > 8 ? sb::kJoinRows : 1; // (rows whose splits a wave requests at once need no other)
  const int64_t each = sb::kJoinRows / waves;
  const dim3 grid((unsigned)((count + each - 1) / each)), block(64 * sb::kJoinRows);
#define SB_JOIN(W)                                                                                                     \
  if (dtype == sb::DT_F32) hipLaunchKernelGGL((sb::join_kernel<sb::DT_F32, W>), grid, block, 0, st, a, count);         \
  else if (dtype == sb::DT_F16) hipLaunchKernelGGL((sb::join_kernel<sb::DT_F16, W>), grid, block, 0, st, a, count);    \
  else hipLaunchKernelGGL((sb::join_kernel<sb::DT_BF16, W>), grid, block, 0, st, a, count)
  if (waves == 1) {
    SB_JOIN(1);
  } else {
    SB_JOIN(sb::kJoinRows);
  }
#undef SB_JOIN
  return hipGetLastError();
}

hipError_t sb_launch_attention_dq_join(const sb::AttnArgs &a, int dtype, hipStream_t st) {
  const sb::FastDiv quads = sb::make_fastdiv((uint32_t)((a.D + 3) / 4));
  const int64_t rows = (int64_t)a.B * a.Hk * a.rows, each = sb::kSumThreads / quads.d;
  const dim3 grid((unsigned)((rows + each - 1) / each)), block(sb::kSumThreads);
  if (dtype == sb::DT_F16) hipLaunchKernelGGL((sb::dq_join_kernel<sb::DT_F16>), grid, block, 0, st, a, quads, rows);
  else hipLaunchKernelGGL((sb::dq_join_kernel<sb::DT_BF16>), grid, block, 0, st, a, quads, rows);
  return hipGetLastError();
}

hipError_t sb_launch_attention_sum(const sb::AttnArgs &a, const sb::AttnHeads *out, int n, int64_t len, int group,
                                   int dtype, hipStream_t st) {
  sb::SumArgs s;
  s.out[0] = out[0];
  s.out[1] = out[n - 1];
  s.part = a.part;
  s.splits = a.splits;
  s.D = a.D;
  s.len = len;
  s.rows = (int64_t)a.B * a.Hk * len;
  s.div_quads = sb::make_fastdiv((uint32_t)((a.D + 3) / 4));
  s.div_group = sb::make_fastdiv((uint32_t)group);
  s.div_Hk = a.div_Hk;
  const int64_t each = sb::kSumThreads / s.div_quads.d;
  const dim3 grid((unsigned)((s.rows + each - 1) / each), (unsigned)n), block(sb::kSumThreads);
  if (dtype == sb::DT_F32) hipLaunchKernelGGL((sb::sum_kernel<sb::DT_F32>), grid, block, 0, st, s);
  else if (dtype == sb::DT_F16) hipLaunchKernelGGL((sb::sum_kernel<sb::DT_F16>), grid, block, 0, st, s);
  else hipLaunchKernelGGL((sb::sum_kernel<sb::DT_BF16>), grid, block, 0, st, s);
  return hipGetLastError();
}
