// sb_attention.h -- launch arguments of the attention kernels, shared by the
// host entry points and the gfx950 kernels.
#pragma once

#include "sb_internal.h"

namespace sb {

// A tensor of heads [B, T, heads, D]: strides in elements, D contiguous.
struct AttnHeads {
  const void *p;
  int64_t b, t, h;
};

// The query heads that share a key head are one list of rows, row q * group + g
// for query q and head g of the group: whatever the group, a tile of rows reads
// a tile of keys once, rows follow the queries (causal order cuts off an end of
// them), and the gradients of a shared key head add up inside one loop.
struct AttnArgs {
  AttnHeads q, k, v, out, dout, dq, dk, dv; // out and the gradients are written (out only forward)
  float *lse;             // [B, heads of q, Lq] natural logarithms (nullptr: not wanted, forward)
  float *delta;           // [B, heads of q, Lq] row sums of dout * out (backward)
  float *peak;            // [units][32 rows] fp16: the largest size of their dS (backward)
  float *part, *part_lse; // partial results of the splits, [splits][units][rows or keys][D] (part_lse: no D)
  float *part_mean, *part_left; // of dq's rows in 16 bits: [splits][units][rows][D] and [splits][units][rows][2]
  const int32_t *q_len, *k_len; // of each sample, or nullptr
  int32_t B, Lq, Lk, Hk, group, D;
  int32_t rows;           // Lq * group
  int32_t causal;
  int32_t tiles, splits;  // of a unit (sample and key head)
  int32_t span;           // keys (rows, for key gradients) of a split, whole tiles
  FastDiv div_group, div_set, div_splits, div_Hk; // (set: the blocks of 8 units)
  uint32_t unit0, units;  // of this launch
  uint32_t blocks;
  int32_t beside;         // tiles of a unit after which the next are put beside them (0: longest first throughout)
  float scale, scale2;    // of the scores, and that times log2(e)
};

constexpr int kAttnWaves = 4;     // waves of a block where there are rows for them
constexpr int64_t kAttnWidth = 256; // longest head

inline int attn_padded(int64_t d) { // head lengths that kernels are built for
  return d <= 32 ? 32 : d <= 64 ? 64 : d <= 96 ? 96 : d <= 128 ? 128 : d <= 160 ? 160 : d <= 192 ? 192 : 256;
}

// Waves of a SIMD that forward's registers are shared out for (blocks of a CU, of
// kAttnWaves): two that take turns at the matrix cores and at the softmax are worth
// more than any register (128 wide, 20280 rows and keys of 12 heads bf16: 5.94 ms for
// one, 2.96 for two); longer heads would spill.
__host__ __device__ constexpr int attn_forward_waves(int elem_bytes, int padded, int waves) {
  if (elem_bytes == 4) return padded <= 32 ? 3 : padded <= 96 || (padded == 128 && waves > 1) ? 2 : 1;
  return padded <= 64 ? 3 : padded <= 160 || (padded == 192 && waves > 1) ? 2 : 1;
}

// heads for which forward has blocks of twice as many waves too
__host__ __device__ constexpr bool attn_wide(int elem_bytes, int padded) {
  return elem_bytes == 2 && padded >= 96 && padded <= 192;
}

// heads for which the gradients' kernels form the next tile's scores while they
// use this one's
__host__ __device__ constexpr bool attn_pipelined(int elem_bytes, int padded) {
  return elem_bytes == 2 && padded <= 192;
}

// keys of a block of the key gradients: 32 a wave, or a pair of waves where a
// head's two halves go to two of them
__host__ __device__ constexpr bool attn_paired(int elem_bytes, int padded) { return padded * elem_bytes > (elem_bytes == 2 ? 384 : 640); }

// dq's kernel that takes any head: two waves to a row (16 bits, whose rows have a second
// sum).  One wave spills: gradient of 4096 tokens of 8 heads of 256 bf16 2.71 ms, 1.32 so; of
// 4 tokens over 4096 keys, heads of 192, 66 us and 47; of 300 tokens of 4 heads of 161 fp16
// 173 and 144; only many rows of 161 to 191 would be faster spilling (2048 tokens of 8 heads
// 547 and 617).
__host__ __device__ constexpr bool attn_dq_paired(int elem_bytes, int padded) { return elem_bytes == 2 && padded >= 192; }

} // namespace sb

// waves: 1, kAttnWaves or (forward, attn_wide) twice that, each with 32 rows of a
// tile; whole: heads of whole 16-byte chunks
hipError_t sb_launch_attention(const sb::AttnArgs &a, int dtype, int waves, hipStream_t st);
hipError_t sb_launch_attention_dq(const sb::AttnArgs &a, int dtype, int waves, int whole, hipStream_t st);
hipError_t sb_launch_attention_dkv(const sb::AttnArgs &a, int dtype, int whole, hipStream_t st);
// joins the splits of the forward pass
hipError_t sb_launch_attention_join(const sb::AttnArgs &a, int dtype, hipStream_t st);
// dq of 16 bits from its splits, and delta with what they leave
hipError_t sb_launch_attention_dq_join(const sb::AttnArgs &a, int dtype, hipStream_t st);
// adds up a.splits splits of n (1 or 2) gradients of the same shape: partial
// results [n][splits][units][len][D] to out[k], rows r of a unit at position
// r / group of head hk * group + r % group
hipError_t sb_launch_attention_sum(const sb::AttnArgs &a, const sb::AttnHeads *out, int n, int64_t len, int group,
                                   int dtype, hipStream_t st);
