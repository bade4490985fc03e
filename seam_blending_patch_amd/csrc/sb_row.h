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

// n elements (any n; fewer than 1 reads nothing) from element e0 of row p,
// zeros after them.
template <int DT> __device__ __forceinline__ Vec<16> load_part(const void *p, int64_t e0, int n) {
  typedef typename El<DT>::bits bits;
  Vec<16> v;
  if (n >= kVec<DT>) {
    const u32x4 q = *reinterpret_cast<const typename El<DT>::vec *>((const bits *)p + e0);
    v.w[0] = q.x; v.w[1] = q.y; v.w[2] = q.z; v.w[3] = q.w;
  } else {
    v.w[0] = v.w[1] = v.w[2] = v.w[3] = 0;
#pragma unroll
    for (int k = 0; k < kVec<DT>; ++k)
      if (k < n) {
        const uint32_t b = ((const bits *)p)[e0 + k];
        if constexpr (DT == DT_F32) v.w[k] = b;
        else v.w[k >> 1] |= b << ((k & 1) * 16);
      }
  }
  return v;
}

// NT: a store past the caches, for results that they could not hold anyway
template <int DT, bool NT = false>
__device__ __forceinline__ void store_part(void *p, int64_t e0, int n, const Vec<16> &v) {
  typedef typename El<DT>::bits bits;
  if (n >= kVec<DT>) {
    const u32x4 q = {v.w[0], v.w[1], v.w[2], v.w[3]};
    typename El<DT>::vec *at = reinterpret_cast<typename El<DT>::vec *>((bits *)p + e0);
    if constexpr (NT) __builtin_nontemporal_store(q, at);
    else *at = q;
  } else {
#pragma unroll
    for (int k = 0; k < kVec<DT>; ++k)
      if (k < n) {
        if constexpr (DT == DT_F32) ((bits *)p)[e0 + k] = v.w[k];
        else ((bits *)p)[e0 + k] = (bits)(v.w[k >> 1] >> ((k & 1) * 16));
      }
  }
}

// A vector of a row that has n elements from there on: where the row is a
// whole number of vectors (no TAIL), it is whole or absent.
template <int DT, bool TAIL> __device__ __forceinline__ Vec<16> load_row(const void *p, int64_t e0, int n) {
  return load_part<DT>(p, e0, TAIL ? n : n > 0 ? kVec<DT> : 0);
}
template <int DT, bool TAIL, bool NT = false>
__device__ __forceinline__ void store_row(void *p, int64_t e0, int n, const Vec<16> &v) {
  store_part<DT, NT>(p, e0, TAIL ? n : n > 0 ? kVec<DT> : 0, v);
}

// N consecutive values of type DT (n of them present, zeros after) as fp32
template <int DT, int N>
__device__ __forceinline__ void load_floats(const void *p, int64_t e0, int n, float *f) {
  static_assert(N % kVec<DT> == 0, "whole vectors");
#pragma unroll
  for (int j = 0; j < N; j += kVec<DT>) unpack<DT, 16>(load_part<DT>(p, e0 + j, n - j), f + j);
}

template <int DT, int N, bool TAIL>
__device__ __forceinline__ void load_floats_row(const void *p, int64_t e0, int n, float *f) {
  load_floats<DT, N>(p, e0, TAIL ? n : n > 0 ? N : 0, f);
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
