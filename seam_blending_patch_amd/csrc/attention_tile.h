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

  static __device__ __forceinline__ u32x4 row_fragment(const char *tile, int r, int u, int h) {
    return *reinterpret_cast<const u32x4 *>(tile + place(r, 2 * u + h));
  }

  // acc += (columns 32 db .. 32 db + 31 of rows r0 .. r0 + 31)^T times the 32 x 32
  // operand `p` (16 result registers of a product; 16-bit: packed in pairs)
  static __device__ __forceinline__ f32x16 column_product(const char *tile, int r0, int db, const uint32_t *p,
                                                          f32x16 acc, int lane) {
    const int h = lane >> 5;
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = r0 + 8 * (i >> 2) + 4 * h + (i & 3);
        const float a = *reinterpret_cast<const float *>(tile + place(r, 8 * db + ((lane & 31) >> 2)) + (lane & 3) * 4);
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a, __uint_as_float(p[i]), acc, 0, 0, 0);
      }
    } else {
      // a transposing read gives lane i of 16 the 16 columns' i-th, of 4 rows
      const int i = lane & 15, c = 4 * db + ((lane >> 4) & 1) * 2 + ((i >> 1) & 1);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        u32x4 a;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = r0 + 16 * t + 8 * half + 4 * h + (i >> 2);
          const auto at = (__attribute__((address_space(3))) char *)tile + place(r, c) + (i & 1) * 8;
          const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)at);
          const uint64_t w = __builtin_bit_cast(uint64_t, v);
          a[2 * half] = (uint32_t)w;
          a[2 * half + 1] = (uint32_t)(w >> 32);
        }
        acc = mma<DT>(a, u32x4{p[4 * t], p[4 * t + 1], p[4 * t + 2], p[4 * t + 3]}, acc);
      }
    }
    return acc;
  }
};

// 16 result registers as the operand of the next product.  16-bit: rounded to
// nearest, so that a product of probabilities (at most 1) or of their gradients
// with 16-bit values adds half a step of each to a sum whose terms have as much.
template <int DT> __device__ __forceinline__ void pack_operand(const float *s, uint32_t *p) {
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = __float_as_uint(s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = narrow2<DT>(f32x2{s[2 * i], s[2 * i + 1]});
  }
}

// One chunk of a row of D elements at p, zeros past its end and for no row.
template <int DT> __device__ __forceinline__ u32x4 load_chunk(const void *p, int64_t row, int c, int D, bool any) {
  const int e = c * kVec<DT>;
  const Vec<16> v = load_part<DT>(p, row + e, any ? D - e : 0);
  return u32x4{v.w[0], v.w[1], v.w[2], v.w[3]};
}

// how the threads of a block share the chunks of a tile
template <int DT, int DP, int ROWS, int THREADS> struct Stage {
  using T = Tile<DT, DP, ROWS>;
  static constexpr int N = (ROWS * T::SC + THREADS - 1) / THREADS; // chunks of a thread
  static constexpr bool kIdle = ROWS * T::SC < THREADS;            // a small tile leaves some threads without one
  static_assert(kIdle || ROWS * T::SC % THREADS == 0, "whole turns");
  u32x4 v[N];
  static __device__ __forceinline__ int row(int k) { return ((int)threadIdx.x + k * THREADS) / T::SC; }
  static __device__ __forceinline__ int chunk() { return (int)threadIdx.x % T::SC; } // the same of every row
  // rows r0 on, those below `end` present; at(r) is a row's first element
  template <class At> __device__ __forceinline__ void load(const void *p, int r0, int end, int D, At at) {
    const int e = chunk() * T::V;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = u32x4{0, 0, 0, 0};
    if (kIdle && row(0) >= ROWS) return;
    if (e + T::V <= D && r0 + ROWS <= end) { // nothing to leave out: requests without a branch between them
#pragma unroll
      for (int k = 0; k < N; ++k)
        v[k] = *reinterpret_cast<const typename El<DT>::vec *>((const typename El<DT>::bits *)p + at(r0 + row(k)) + e);
    } else if (e < D) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (r0 + row(k) < end) v[k] = load_chunk<DT>(p, at(r0 + row(k)), chunk(), D, true);
    }
  }
  __device__ __forceinline__ void store(char *tile) const {
    if ((T::kChunks == T::SC || chunk() < T::kChunks) && !(kIdle && row(0) >= ROWS)) {
#pragma unroll
      for (int k = 0; k < N; ++k) *reinterpret_cast<u32x4 *>(tile + T::place(row(k), chunk())) = v[k];
    }
  }
};

// a block's work: its unit (sample and key head), its tile of the unit's rows or
// keys and its split of the other side.  Blocks go to the 8 XCDs in turn; each
// of those takes a run of consecutive work, so that the blocks which read the
// same keys (rows) share an L2.
struct Work {
  uint32_t unit;
  int b, hk, tile, split;
};
__device__ __forceinline__ Work work_of(const AttnArgs &a) {
  const uint32_t id = blockIdx.x, xcd = id & 7, per = a.blocks >> 3, more = a.blocks & 7;
  const uint32_t w = xcd * per + min(xcd, more) + (id >> 3);
  const uint32_t s = fdiv(w, a.div_tiles), u = fdiv(s, a.div_splits);
  Work k;
  k.tile = (int)(w - s * a.div_tiles.d);
  k.split = (int)(s - u * a.div_splits.d);
  k.unit = a.unit0 + u;
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
