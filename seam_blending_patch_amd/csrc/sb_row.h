// sb_row.h -- rows of storage elements read and written in 16-byte vectors at
// any element alignment, and sums over the lanes that share a row.
#pragma once

#include "sb_vec.h"

namespace sb {

// 16 bytes at the alignment of one element: global memory takes vector
// accesses at any address the element type allows (the compiler emits the
// same global_load_dwordx4 / store as for aligned ones), so rows of odd length
// and views at odd offsets need no path of their own.
typedef u32x4 u32x4_el2 __attribute__((aligned(2)));
typedef u32x4 u32x4_el4 __attribute__((aligned(4)));
template <int DT> struct El { typedef u32x4_el2 vec; typedef uint16_t bits; };
template <> struct El<DT_F32> { typedef u32x4_el4 vec; typedef uint32_t bits; };

// elements per 16-byte vector
template <int DT> constexpr int kVec = 16 / Elem<DT>::bytes;

// A vector cut short, in pieces of 4, 2 and 1 elements (2 and 1 of fp32): three
// accesses at most, where one an element would be seven.
typedef uint32_t u32x2_el2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x2_el4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32_el2 __attribute__((aligned(2)));

// (selected by value: among array elements `?:` would select an address, and the
// array would live in memory)
__device__ __forceinline__ uint32_t pick(bool c, uint32_t yes, uint32_t no) { return c ? yes : no; }

template <int DT> __device__ __forceinline__ void load_cut(const typename El<DT>::bits *p, int n, Vec<16> &v) {
  if constexpr (DT == DT_F32) {
    u32x2_el4 two = {0, 0};
    uint32_t one = 0;
    if (n & 2) two = *reinterpret_cast<const u32x2_el4 *>(p);
    if (n & 1) one = p[n & 2];
    v.w[0] = pick(n & 2, two.x, one);
    v.w[1] = two.y;
    v.w[2] = pick(n & 2, one, 0);
    v.w[3] = 0;
  } else {
    u32x2_el2 four = {0, 0};
    uint32_t two = 0, one = 0;
    if (n & 4) four = *reinterpret_cast<const u32x2_el2 *>(p);
    if (n & 2) two = *reinterpret_cast<const u32_el2 *>(p + (n & 4));
    if (n & 1) one = p[n & 6];
    const uint32_t a = pick(n & 2, two, one), b = pick(n & 2, one, 0);
    v.w[0] = pick(n & 4, four.x, a);
    v.w[1] = pick(n & 4, four.y, b);
    v.w[2] = pick(n & 4, a, 0);
    v.w[3] = pick(n & 4, b, 0);
  }
}

template <int DT> __device__ __forceinline__ void store_cut(typename El<DT>::bits *p, int n, const Vec<16> &v) {
  if constexpr (DT == DT_F32) {
    const uint32_t one = pick(n & 2, v.w[2], v.w[0]);
    if (n & 2) *reinterpret_cast<u32x2_el4 *>(p) = u32x2_el4{v.w[0], v.w[1]};
    if (n & 1) p[n & 2] = one;
  } else {
    const uint32_t a = pick(n & 4, v.w[2], v.w[0]), b = pick(n & 4, v.w[3], v.w[1]);
    if (n & 4) *reinterpret_cast<u32x2_el2 *>(p) = u32x2_el2{v.w[0], v.w[1]};
    if (n & 2) *reinterpret_cast<u32_el2 *>(p + (n & 4)) = a;
    if (n & 1) p[n & 6] = (uint16_t)pick(n & 2, b, a);
  }
}

// n elements (any n; fewer than 1 reads nothing) from element e0 of row p,
// zeros after them.
template <int DT> __device__ __forceinline__ Vec<16> load_part(const void *p, int64_t e0, int n) {
  const auto *at = (const typename El<DT>::bits *)p + e0;
  Vec<16> v;
  v.w[0] = v.w[1] = v.w[2] = v.w[3] = 0;
  if (n >= kVec<DT>) {
    const u32x4 q = *reinterpret_cast<const typename El<DT>::vec *>(at);
    v.w[0] = q.x; v.w[1] = q.y; v.w[2] = q.z; v.w[3] = q.w;
  } else if (n > 0) {
    load_cut<DT>(at, n, v);
  }
  return v;
}

// NT: a store past the caches, for results that they could not hold anyway
template <int DT, bool NT = false>
__device__ __forceinline__ void store_part(void *p, int64_t e0, int n, const Vec<16> &v) {
  auto *at = (typename El<DT>::bits *)p + e0;
  if (n >= kVec<DT>) {
    const u32x4 q = {v.w[0], v.w[1], v.w[2], v.w[3]};
    if constexpr (NT) __builtin_nontemporal_store(q, reinterpret_cast<typename El<DT>::vec *>(at));
    else *reinterpret_cast<typename El<DT>::vec *>(at) = q;
  } else if (n > 0) {
    store_cut<DT>(at, n, v);
  }
}

// What is known of a vector of a row: its row covers it, it may lie past the
// row's end, or it may be cut by that.
enum Cover : int { WHOLE, WHOLE_OR_NONE, CUT };

// The vector of a row of D elements from element e on.  One that may be cut is
// requested V elements before the row's end where it would pass that, so that
// every lane's request is one access and none diverges, and moved into place
// when it is used (rows shorter than a vector go in pieces).
template <int DT, Cover C> __device__ __forceinline__ Vec<16> request_row(const void *p, int64_t base, int e, int D) {
  constexpr int V = kVec<DT>;
  if constexpr (C == WHOLE) return load_part<DT>(p, base + e, V);
  else if constexpr (C == WHOLE_OR_NONE) return load_part<DT>(p, base + e, D > e ? V : 0);
  else if (D >= V) return load_part<DT>(p, base + min(e, D - V), V);
  else return load_part<DT>(p, base + e, D - e);
}

// the first `bits` (1 or more) of 128 dropped, zeros after the others
__device__ __forceinline__ void shift_down(Vec<16> &v, int bits) {
  uint64_t lo = v.w[0] | (uint64_t)v.w[1] << 32, hi = v.w[2] | (uint64_t)v.w[3] << 32;
  if (bits >= 64) {
    lo = bits >= 128 ? 0 : hi >> (bits & 63);
    hi = 0;
  } else {
    lo = lo >> bits | hi << (64 - bits);
    hi >>= bits;
  }
  v.w[0] = (uint32_t)lo; v.w[1] = (uint32_t)(lo >> 32);
  v.w[2] = (uint32_t)hi; v.w[3] = (uint32_t)(hi >> 32);
}
template <int DT, Cover C> __device__ __forceinline__ void settle_row(Vec<16> &v, int e, int D) {
  if constexpr (C == CUT) {
    const int before = e + kVec<DT> - D; // elements that the request began too early
    if (before > 0 && D >= kVec<DT>) shift_down(v, before * Elem<DT>::bytes * 8);
  }
}

template <int DT, Cover C, bool NT = false>
__device__ __forceinline__ void store_row(void *p, int64_t base, int e, int D, const Vec<16> &v) {
  store_part<DT, NT>(p, base + e, C == WHOLE ? kVec<DT> : C == CUT ? D - e : D > e ? kVec<DT> : 0, v);
}

// N consecutive values of a row of weights (a multiple of a vector's) as fp32
template <int DT, int N, Cover C> __device__ __forceinline__ void load_weights(const void *p, int e, int D, float *f) {
  static_assert(N % kVec<DT> == 0, "whole vectors");
  Vec<16> v[N / kVec<DT>];
#pragma unroll
  for (int j = 0; j < N / kVec<DT>; ++j) v[j] = request_row<DT, C>(p, 0, e + j * kVec<DT>, D);
#pragma unroll
  for (int j = 0; j < N / kVec<DT>; ++j) {
    settle_row<DT, C>(v[j], e + j * kVec<DT>, D);
    unpack<DT, 16>(v[j], f + j * kVec<DT>);
  }
}

// N consecutive values of type DT (n of them present, zeros after) as fp32
template <int DT, int N>
__device__ __forceinline__ void load_floats(const void *p, int64_t e0, int n, float *f) {
  static_assert(N % kVec<DT> == 0, "whole vectors");
#pragma unroll
  for (int j = 0; j < N; j += kVec<DT>) unpack<DT, 16>(load_part<DT>(p, e0 + j, n - j), f + j);
}

// One value per lane summed over every aligned group of LANES lanes, returned
// in each of them: butterflies over DPP quad permutes and row mirrors (after a
// level all lanes of a group hold the same bits, so the mirrored lane stands
// for the exchanged one), then gfx950's row and half-wave swaps.  Additions
// commute, so every lane of the group ends with the same bits.  All 64 lanes
// have to be active.
template <int CTRL> __device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (LANES >= 2) v = dpp_add<0xB1>(v);   // quad_perm [1,0,3,2]
  if constexpr (LANES >= 4) v = dpp_add<0x4E>(v);   // quad_perm [2,3,0,1]
  if constexpr (LANES >= 8) v = dpp_add<0x141>(v);  // row_half_mirror
  if constexpr (LANES >= 16) v = dpp_add<0x140>(v); // row_mirror
  if constexpr (LANES >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if constexpr (LANES >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return v;
}

// K values summed over every group of LANES threads of a block of THREADS,
// returned in each of the group's threads.  Up to 64 lanes no memory is used;
// wider groups exchange their waves' sums through `lds`, whose halves are
// taken in turn (`turn` flips on every call): a wave may still read one while
// another writes the other, so one barrier a sum is enough.
template <int LANES, int K, int N>
__device__ __forceinline__ void group_sum(float (&v)[K], float (&lds)[2][N], int &turn) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lanes_sum<(LANES < 64 ? LANES : 64)>(v[k]);
  if constexpr (LANES > 64) {
    constexpr int W = LANES / 64; // waves of a group
    const int wave = threadIdx.x >> 6;
    float *s = lds[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) s[wave * K + k] = v[k];
    }
    __syncthreads();
    s += wave / W * W * K;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = s[k];
#pragma unroll
    for (int w = 1; w < W; ++w) {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += s[w * K + k];
    }
  }
}

} // namespace sb
