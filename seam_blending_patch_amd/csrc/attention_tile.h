// attention_tile.h -- tiles of heads in LDS and matrix-core products of 32 x 32
// tiles, as the attention kernels use them.
//
// Everything is built on products C += A B with 32 x 32 results: a lane holds
// column n = lane % 32 of C, rows 8 (i / 4) + 4 h + i % 4 in its 16 registers,
// h = lane / 32.  16-bit products take 16 terms (lane: row or column lane % 32,
// terms 8 h .. 8 h + 7), fp32 ones 2 (term h).  The terms of a product may come
// in any order as long as A and B agree, which is used twice:
//  - a "row fragment" u is the 16 bytes at chunk 2 u + h of a row, whatever the
//    type: 8 terms of one 16-bit product, or a term each of 4 fp32 products;
//  - the result registers of one product are, converted and packed, an operand
//    of the next without moving between lanes: registers 8 t .. 8 t + 7 hold
//    rows 16 t + 4 h + {0..3} and 16 t + 8 + 4 h + {0..3}, and the other
//    operand's fragment takes those rows of its tile.
#pragma once

#include <type_traits>
#include <utility>

#include "sb_attention.h"
#include "sb_row.h"

namespace sb {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kInf = __builtin_inff();

// C += A B over one row fragment of each
template <int DT> __device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[j]), __uint_as_float(b[j]), c, 0, 0, 0);
  } else if constexpr (DT == DT_F16) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  } else {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                0);
  }
  return c;
}

// A tile of ROWS rows of heads of up to DP elements in LDS: rows of SC chunks of
// 16 bytes (a power of two), chunk c of row r at place c ^ mix(r).  The mix
// spreads both ways of reading over the banks: one chunk of 16 or 32 consecutive
// rows, and the same 64 bytes of 4 consecutive rows.
template <int DT, int DP, int ROWS> struct Tile {
  static constexpr int V = kVec<DT>;
  static constexpr int kChunks = DP / V;          // of a row
  static constexpr int SC = kChunks <= 4 ? 4 : kChunks <= 8 ? 8 : kChunks <= 16 ? 16 : kChunks <= 32 ? 32 : 64;
  static constexpr int kFrags = kChunks / 2;      // row fragments
  static constexpr int kBytes = ROWS * SC * 16;
  static __device__ __forceinline__ int mix(int r) {
    if constexpr (SC >= 16) return ((r & 3) << 2) | ((r >> 2) & 3);
    else if constexpr (SC == 8) return ((r & 2) << 1) | ((r >> 2) & 3);
    else return (r >> 2) & 3;
  }
  static __device__ __forceinline__ int place(int r, int c) { return (r * SC + (c ^ mix(r))) * 16; }

  // Places as a lane's own offset, in which only bits below a row's length still
  // change, by exclusive or with what the loops count: no address arithmetic is
  // left but that, and whole rows are constant offsets.  `tile` is an offset too.
  //
  // row fragment u of row r0 + lane % 32:
  static __device__ __forceinline__ int row_place(int lane) { return place(lane & 31, lane >> 5); }
  static __device__ __forceinline__ u32x4 row_fragment(const char *lds, int place, int r0, int u) {
    return *reinterpret_cast<const u32x4 *>(lds + (place ^ (u << 5)) + r0 * (SC * 16));
  }
  // columns 32 db .. 32 db + 31 of the rows that column_product takes
  static __device__ __forceinline__ int column_place(int lane) {
    const int h = lane >> 5;
    if constexpr (DT == DT_F32) return place(4 * h, (lane & 31) >> 2) + (lane & 3) * 4;
    const int i = lane & 15; // of 16 lanes, which read the 4 columns i % 4 of row i / 4 and get column i of 4 rows
    return place(4 * h + (i >> 2), ((lane >> 4) & 1) * 2 + ((i >> 1) & 1)) + (i & 1) * 8;
  }

  // 16-bit: the fragment of those columns for terms 16 t .. 16 t + 15 of rows r0 on
  static __device__ __forceinline__ u32x4 column_fragment(const char *lds, int place, int r0, int db, int t) {
    u32x4 a;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = 16 * t + 8 * half;
      const auto at = (__attribute__((address_space(3))) const char *)lds + (place ^ (mix(r) << 4) ^ (db << 6))
                      + (r0 + r) * (SC * 16);
      const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)at);
      const uint64_t w = __builtin_bit_cast(uint64_t, v);
      a[2 * half] = (uint32_t)w;
      a[2 * half + 1] = (uint32_t)(w >> 32);
    }
    return a;
  }

  // acc += (columns 32 db .. of rows r0 .. r0 + 31)^T times the 32 x 32 operand `p`
  // (16 result registers of a product; 16-bit: packed in pairs)
  static __device__ __forceinline__ f32x16 column_product(const char *lds, int place, int r0, int db,
                                                          const uint32_t *p, f32x16 acc) {
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = 8 * (i >> 2) + (i & 3);
        const float a = *reinterpret_cast<const float *>(lds + (place ^ (mix(r) << 4) ^ (db << 7)) + (r0 + r) * (SC * 16));
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a, __uint_as_float(p[i]), acc, 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 2; ++t)
        acc = mma<DT>(column_fragment(lds, place, r0, db, t), u32x4{p[4 * t], p[4 * t + 1], p[4 * t + 2], p[4 * t + 3]},
                      acc);
    }
    return acc;
  }
};

// Products whose fragments are read from LDS AHEAD of them: read(i) gives the
// fragment of step i, use(i, fragment) its product.  The order is kept as written.
// (One call a step, not a loop: the unrolled whole would pass the compiler's limit
// for one, and what a step counts with has to be constant.)
template <int I, int N, int AHEAD, class Read, class Use>
__device__ __forceinline__ void in_order_step(u32x4 (&f)[AHEAD], Read &read, Use &use) {
  use(I, f[I % AHEAD]);
  if constexpr (I + AHEAD < N) f[I % AHEAD] = read(I + AHEAD);
  __builtin_amdgcn_sched_barrier(0);
}
template <int N, int AHEAD, class Read, class Use, int... I>
__device__ __forceinline__ void in_order_steps(std::integer_sequence<int, I...>, u32x4 (&f)[AHEAD], Read &read, Use &use) {
  (in_order_step<I, N, AHEAD>(f, read, use), ...);
}
template <int N, int AHEAD, class Read, class Use> __device__ __forceinline__ void in_order(Read read, Use use) {
  u32x4 f[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD && i < N; ++i) f[i] = read(i);
  __builtin_amdgcn_sched_barrier(0);
  in_order_steps<N, AHEAD>(std::make_integer_sequence<int, N>{}, f, read, use);
}

// 16 result registers as the operand of the next product.  16-bit: rounded to
// nearest, so that a product of probabilities (times a power of two) or of their
// gradients with 16-bit values adds half a step of each to a sum whose terms have as
// much.
template <int DT> __device__ __forceinline__ void pack_operand(const float *s, uint32_t *p) {
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = __float_as_uint(s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = narrow2<DT>(f32x2{s[2 * i], s[2 * i + 1]});
  }
}

template <int DT> __device__ __forceinline__ uint32_t pack_pair(const float *s) { return narrow2<DT>(f32x2{s[0], s[1]}); }

// c + the two values of a packed pair
template <int DT> __device__ __forceinline__ float pair_sum(uint32_t w, float c) {
  if constexpr (DT == DT_F16)
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, w), __builtin_bit_cast(f16x2, 0x3C003C00u), c, false);
  else
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, 0x3F803F80u), c,
                                           false);
}

// One chunk of a row of D elements at p, zeros past its end and for no row.
template <int DT> __device__ __forceinline__ u32x4 load_chunk(const void *p, int64_t row, int c, int D, bool any) {
  const int e = c * kVec<DT>;
  const Vec<16> v = load_part<DT>(p, row + e, any ? D - e : 0);
  return u32x4{v.w[0], v.w[1], v.w[2], v.w[3]};
}

// How the threads of a block share the chunks of a tile: TURNS of them (all, or as
// many as are to be in registers at a time) from turn k0 on.
template <int DT, int DP, int ROWS, int THREADS> struct Share {
  using T = Tile<DT, DP, ROWS>;
  static constexpr int N = (ROWS * T::SC + THREADS - 1) / THREADS; // chunks of a thread
  static constexpr bool kIdle = ROWS * T::SC < THREADS;            // a small tile leaves some threads without one
  static_assert(kIdle || ROWS * T::SC % THREADS == 0, "whole turns");
  static __device__ __forceinline__ int row(int k) { return ((int)threadIdx.x + k * THREADS) / T::SC; }
  static __device__ __forceinline__ int chunk() { return (int)threadIdx.x % T::SC; } // the same of every row
};
template <int DT, int DP, int ROWS, int THREADS, int TURNS = Share<DT, DP, ROWS, THREADS>::N>
struct Stage : Share<DT, DP, ROWS, THREADS> {
  using S = Share<DT, DP, ROWS, THREADS>;
  using T = typename S::T;
  using S::chunk;
  using S::row;
  u32x4 v[TURNS];
  // rows r0 on, those below `end` present; at(r) is a row's first element
  template <class At> __device__ __forceinline__ void load(const void *p, int r0, int end, int D, At at, int k0 = 0) {
    const int e = chunk() * T::V;
#pragma unroll
    for (int k = 0; k < TURNS; ++k) v[k] = u32x4{0, 0, 0, 0};
    if (S::kIdle && row(0) >= ROWS) return;
    if (e + T::V <= D && r0 + ROWS <= end) { // nothing to leave out: requests without a branch between them
#pragma unroll
      for (int k = 0; k < TURNS; ++k)
        v[k] = *reinterpret_cast<const typename El<DT>::vec *>((const typename El<DT>::bits *)p + at(r0 + row(k0 + k)) + e);
    } else if (e < D) {
#pragma unroll
      for (int k = 0; k < TURNS; ++k)
        if (r0 + row(k0 + k) < end) v[k] = load_chunk<DT>(p, at(r0 + row(k0 + k)), chunk(), D, true);
    }
  }
  __device__ __forceinline__ void store(char *tile, int k0 = 0) const {
    if ((T::kChunks == T::SC || chunk() < T::kChunks) && !(S::kIdle && row(0) >= ROWS)) {
#pragma unroll
      for (int k = 0; k < TURNS; ++k) *reinterpret_cast<u32x4 *>(tile + T::place(row(k0 + k), chunk())) = v[k];
    }
  }
};
// Tiles of consecutive rows of whole chunks (D a multiple of one), one after the
// other, at a stride: a thread's place moves by a tile, nothing is multiplied on
// the way.  Rows past the end are zeros (what is requested in their place is the
// last row); chunks past D are not stored: clear_tiles puts zeros there once.
template <int DT, int DP, int ROWS, int THREADS> struct RowStage {
  using S = Share<DT, DP, ROWS, THREADS>;
  using T = typename S::T;
  static constexpr int N = S::N;
  typedef typename El<DT>::bits bits;
  u32x4 v[N];
  const bits *at;     // of this thread, in the next tile
  int64_t stride;
  bool any;           // the thread has a chunk of every row
  __device__ __forceinline__ void start(const void *p, int64_t base, int64_t row_stride, int r0, int D) {
    any = S::chunk() * T::V < D && !(S::kIdle && S::row(0) >= ROWS);
    stride = row_stride;
    at = (const bits *)p + base + (int64_t)(r0 + (any ? S::row(0) : 0)) * stride + (any ? S::chunk() * T::V : 0);
  }
  __device__ __forceinline__ void load(int r0, int end) { // rows r0 on, those below `end` (r0 is one) present
    const int left = end - r0;
    if (left >= ROWS) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        v[k] = *reinterpret_cast<const typename El<DT>::vec *>(at + k * (THREADS / T::SC) * stride);
    } else {
      const int mine = any ? S::row(0) : 0; // (at's row)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int r = mine + k * (THREADS / T::SC);
        const u32x4 w = *reinterpret_cast<const typename El<DT>::vec *>(at + (int64_t)(min(r, left - 1) - mine) * stride);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k][i] = r < left ? w[i] : 0;
      }
    }
    at += ROWS * stride;
  }
  __device__ __forceinline__ void store(char *lds) const {
    if (any) {
#pragma unroll
      for (int k = 0; k < N; ++k) *reinterpret_cast<u32x4 *>(lds + T::place(S::row(k), S::chunk())) = v[k];
    }
  }
};
// A barrier for LDS alone: what is on its way from memory stays on its way.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// zeros in `bytes` of LDS where heads are shorter than what the kernel is built for
template <int THREADS> __device__ __forceinline__ void clear_tiles(char *lds, int bytes, bool shorter) {
  if (shorter) {
    for (int i = threadIdx.x * 16; i < bytes; i += THREADS * 16) *reinterpret_cast<u32x4 *>(lds + i) = u32x4{0, 0, 0, 0};
    __syncthreads();
  }
}

// a whole tile now, a few chunks of a thread at a time
template <int DT, int DP, int ROWS, int THREADS, class At>
__device__ __forceinline__ void stage_tile(char *tile, const void *p, int r0, int end, int D, At at) {
  constexpr int N = Share<DT, DP, ROWS, THREADS>::N, TURNS = N < 8 ? N : 8;
#pragma unroll 1
  for (int k0 = 0; k0 < N; k0 += TURNS) {
    Stage<DT, DP, ROWS, THREADS, TURNS> st;
    st.load(p, r0, end, D, at, k0);
    st.store(tile, k0);
  }
}

// A block's work: its unit (sample and key head), its tile of the unit's rows or
// keys and its split of the other side.  Blocks go to the 8 XCDs in turn: units in
// sets of 8, a unit of them to each, so that the blocks that read the same keys
// (rows) share an L2.  (One by one, their tiles over all XCDs, is no better where
// lengths differ: 3 samples of 1537, 769 and 0 tokens, 16 heads of 64, backward 108 us
// against 104.)  In a unit the tiles with most to do come first: causal order leaves
// the last rows, or the first keys, the most.
struct Work {
  uint32_t unit;
  int b, hk, tile, split;
};
template <bool LAST_FIRST> __device__ __forceinline__ Work work_of(const AttnArgs &a) {
  const uint32_t set = fdiv(blockIdx.x, a.div_set), first = set * 8, in = blockIdx.x - set * a.div_set.d;
  const uint32_t of = min(8u, a.units - first), rest = in / of;
  Work k;
  k.unit = a.unit0 + first + (in - rest * of);
  k.tile = (int)fdiv(rest, a.div_splits);
  k.split = (int)rest - k.tile * (int)a.div_splits.d;
  if (a.beside && k.tile >= a.beside) { // the second tiles of the CUs get longer as the first get shorter
    const int over = max(a.tiles - 2 * a.beside, 0); // (the shortest of all, for whoever is done first)
    k.tile = k.tile < 2 * a.beside ? a.tiles - 1 - over - (k.tile - a.beside) : a.tiles - over + (k.tile - 2 * a.beside);
  }
  if (LAST_FIRST) k.tile = a.tiles - 1 - k.tile;
  k.b = (int)fdiv(k.unit, a.div_Hk);
  k.hk = (int)(k.unit - (uint32_t)k.b * a.div_Hk.d);
  return k;
}

// lengths of a sample, within its tensors
__device__ __forceinline__ int length_of(const int32_t *len, int b, int most) {
  return len ? min(max(len[b], 0), most) : most;
}

// element offset of a packed row
__device__ __forceinline__ int64_t row_at(const AttnHeads &x, const AttnArgs &a, int b, int hk, int r) {
  const int q = (int)fdiv((uint32_t)r, a.div_group), g = r - q * a.group;
  return b * x.b + q * x.t + (int64_t)(hk * a.group + g) * x.h;
}
// index of a packed row in [B, heads, Lq]
__device__ __forceinline__ int64_t stat_at(const AttnArgs &a, int b, int hk, int r) {
  const int q = (int)fdiv((uint32_t)r, a.div_group), g = r - q * a.group;
  return ((int64_t)b * a.Hk * a.group + hk * a.group + g) * a.Lq + q;
}

// the sum and the maximum of a lane's value and the other half-wave's
__device__ __forceinline__ float half_sum(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
__device__ __forceinline__ float half_max(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// 4 values to elements e .. e + 3 of a tensor, the first n of them
typedef float f32x4v __attribute__((ext_vector_type(4)));
template <int DT> __device__ __forceinline__ void store_four(void *p, int64_t e, int n, f32x4v f) {
  if constexpr (DT == DT_F32) {
    Vec<16> v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.w[i] = __float_as_uint(f[i]);
    store_part<DT>(p, e, n, v);
  } else {
    uint16_t *to = (uint16_t *)p + e;
    const uint32_t lo = narrow2<DT>(f32x2{f[0], f[1]}), hi = narrow2<DT>(f32x2{f[2], f[3]});
    if (n >= 4) {
      *reinterpret_cast<u32x2_el2 *>(to) = u32x2_el2{lo, hi};
    } else if (n > 0) {
      to[0] = (uint16_t)lo;
      if (n > 1) to[1] = (uint16_t)(lo >> 16);
      if (n > 2) to[2] = (uint16_t)hi;
    }
  }
}

// A lane's results of a transposed 32-column block (rows d = 32 db + 8 (i / 4) +
// 4 h + i % 4 of its column) to the row of D elements at `at`
template <int DT> __device__ __forceinline__ void store_column(void *p, int64_t at, int db, int h, int D, f32x16 acc,
                                                               float by) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int d = 32 * db + 8 * j + 4 * h;
    store_four<DT>(p, at + d, D - d,
                   f32x4v{acc[4 * j] * by, acc[4 * j + 1] * by, acc[4 * j + 2] * by, acc[4 * j + 3] * by});
  }
}

} // namespace sb
