// attention.cpp -- host side of attention_forward and attention_backward:
// argument checks, how the work is cut into blocks and splits, the workspace's
// layout.  No device memory is allocated and the stream is never synchronised.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "sb_attention.h"
#include "sb_host.h"
#include "sb_strided.h"

using sb::failf;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30; // packed rows, and keys times the group: 32-bit indices
constexpr int64_t kMaxHeads = 1 << 12;
constexpr int64_t kMaxUnits = (int64_t)1 << 30; // samples times key heads
constexpr int kMaxSplits = 64;                  // a lane of the joining wave has one

int read_shape(const int64_t *shape, int dtype, sb::AttnArgs &a) {
  if (!sb::known_dtype(dtype)) return failf(SB_EARG, "unknown dtype %d", dtype);
  if (!shape) return failf(SB_EARG, "null shape");
  const int64_t B = shape[0], Lq = shape[1], Lk = shape[2], Hq = shape[3], Hk = shape[4], D = shape[5];
  if (B < 0 || Lq < 0 || Lk < 0) return failf(SB_EARG, "negative extent");
  if (Hq < 1 || Hk < 1 || Hq % Hk != 0)
    return failf(SB_EARG, "query heads (%lld) must be a multiple of the key heads (%lld)", (long long)Hq, (long long)Hk);
  if (Hq > kMaxHeads) return failf(SB_EGEOM, "more than %lld heads", (long long)kMaxHeads);
  if (D < 1 || D > sb::kAttnWidth)
    return failf(SB_EGEOM, "head length must be in 1..%lld (got %lld)", (long long)sb::kAttnWidth, (long long)D);
  const int64_t group = Hq / Hk;
  if (Lq >= kMaxRows || Lk >= kMaxRows || Lq * group >= kMaxRows || Lk * group >= kMaxRows)
    return failf(SB_EGEOM, "lengths times the query heads of a key head must be below 2^30");
  if (B >= kMaxUnits || B * Hk >= kMaxUnits) return failf(SB_EGEOM, "2^30 samples times key heads or more");
  std::memset(&a, 0, sizeof a);
  a.B = (int32_t)B;
  a.Lq = (int32_t)Lq;
  a.Lk = (int32_t)Lk;
  a.Hk = (int32_t)Hk;
  a.group = (int32_t)group;
  a.D = (int32_t)D;
  a.rows = (int32_t)(Lq * group);
  a.div_group = sb::make_fastdiv((uint32_t)group);
  a.div_Hk = sb::make_fastdiv((uint32_t)Hk);
  return SB_OK;
}

int check_scale(float scale, sb::AttnArgs &a) {
  if (!(scale > 0.0f && scale < __builtin_inff())) return failf(SB_EARG, "scale must be positive and finite");
  a.scale = scale;
  a.scale2 = (float)((double)scale * 1.4426950408889634);
  if (!(a.scale2 < __builtin_inff()) || a.scale2 < 1e-30f) return failf(SB_EARG, "scale must be in 1e-30..2e38");
  return SB_OK;
}

int check_lengths(const int32_t *q_len, const int32_t *k_len, sb::AttnArgs &a) {
  if (!sb::aligned(q_len, 4) || !sb::aligned(k_len, 4))
    return failf(SB_EARG, "lengths must be aligned to their element size");
  a.q_len = q_len;
  a.k_len = k_len;
  return SB_OK;
}

// one tensor [B, T, heads, D]
struct Heads {
  const char *name;
  const void *p;
  sb::Strided s;
};

int read_heads(const char *name, const void *p, const int64_t *stride, const sb::AttnArgs &a, int64_t length,
               int64_t heads, int dtype, sb::AttnHeads &out, Heads &h) {
  h.name = name;
  h.p = p;
  if (a.B == 0 || length == 0) { // nothing to read or write
    out = sb::AttnHeads{nullptr, 0, 0, 0};
    h.p = nullptr;
    return SB_OK;
  }
  if (!p || !stride) return failf(SB_EARG, "null %s or strides of %s", name, name);
  for (int k = 0; k < 3; ++k)
    if (stride[k] < 0 || stride[k] >= sb::kMaxStride)
      return failf(SB_EGEOM, "strides of %s must be in 0..2^40 elements", name);
  if (!sb::aligned(p, sb::elem_bytes(dtype))) return failf(SB_EARG, "%s is not aligned to its element size", name);
  h.s.run = a.D;
  h.s.add(a.B, stride[0]);
  h.s.add(length, stride[1]);
  h.s.add(heads, stride[2]);
  if (h.s.span() >= sb::kMaxSpan) return failf(SB_EGEOM, "%s spans 2^52 elements or more", name);
  out = sb::AttnHeads{p, stride[0], stride[1], stride[2]};
  return SB_OK;
}

// an output has to hold every element once and to share none with `other`
int check_apart(const Heads &out, const Heads &other, int dtype) {
  if (!out.p || !other.p) return SB_OK;
  const int64_t eb = sb::elem_bytes(dtype), bytes = (int64_t)((uintptr_t)out.p - (uintptr_t)other.p);
  if (bytes % eb != 0 || sb::can_overlap(other.s, out.s, bytes / eb))
    return failf(SB_EARG, "%s overlaps %s", out.name, other.name);
  return SB_OK;
}
int check_distinct(const Heads &out) {
  return out.p && !out.s.distinct() ? failf(SB_EARG, "%s overlaps itself", out.name) : SB_OK;
}

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// How a kernel's work is cut: blocks of `waves` waves with 32 rows (keys) each, the
// other side in splits where that alone does not fill the chip (causal gradients
// into more, for their longest tiles are twice the mean).
struct Plan {
  int waves;
  int64_t tiles, splits, span;
};

Plan cut(int64_t units, int64_t own, int64_t per_block, int64_t along, int waves, int64_t want, int64_t least) {
  Plan p;
  p.waves = waves;
  p.tiles = (own + per_block - 1) / per_block;
  const int64_t blocks = std::max<int64_t>(1, units * p.tiles);
  const int64_t most = std::min<int64_t>(kMaxSplits, (along + least - 1) / least);
  p.splits = blocks * 2 > want ? 1 : std::max<int64_t>(1, std::min(most, want / blocks));
  p.span = std::max<int64_t>(64, up((along + p.splits - 1) / p.splits, 64));
  p.splits = std::max<int64_t>(1, (along + p.span - 1) / p.span);
  return p;
}

bool whole_chunks(const sb::AttnArgs &a, int dtype) { return a.D % (16 / sb::elem_bytes(dtype)) == 0; }

Plan plan_rows(const sb::AttnArgs &a, int dtype, bool forward, bool causal, bool lengths) {
  const int64_t cus = sb_cu_count(), want = !forward && causal ? 3 * cus : cus, units = (int64_t)a.B * a.Hk;
  const int eb = sb::elem_bytes(dtype), padded = sb::attn_padded(a.D), wide = 2 * sb::kAttnWaves;
  const bool whole = whole_chunks(a, dtype);
  // Single tokens: a wave to a block, as many splits as keep the memory busy; twice
  // as many where lengths leave some of them empty (8 tokens over 16384, 14044, ... 0
  // keys, 32 heads of 128 in 8 groups bf16, the same inputs again, 61.9 us with 16 waves
  // a CU, 69.0 with 8 (72 with 16 where inputs change and none is in the caches);
  // 32 over 4096 keys each 118 and 108).
  if (a.rows <= 32) return cut(units, a.rows, 32, a.Lk, 1, (lengths ? 16 : 8) * cus, 128);
  if (forward && whole && sb::attn_wide(eb, padded) && units * ((a.rows + 32 * wide - 1) / (32 * wide)) >= 2 * cus)
    return cut(units, a.rows, 32 * wide, a.Lk, wide, 1, a.Lk + 1);
  const bool paired = !forward && !(whole && sb::attn_pipelined(eb, padded)) && sb::attn_dq_paired(eb, padded);
  return cut(units, a.rows, 32 * sb::kAttnWaves / (paired ? 2 : 1), a.Lk, sb::kAttnWaves, want, 512);
}

Plan plan_keys(const sb::AttnArgs &a, int dtype, bool causal) {
  const int64_t cus = sb_cu_count(), units = (int64_t)a.B * a.Hk;
  const bool paired = sb::attn_paired(sb::elem_bytes(dtype), sb::attn_padded(a.D));
  return cut(units, a.Lk, 32 * sb::kAttnWaves / (paired ? 2 : 1), a.rows, sb::kAttnWaves, causal ? 3 * cus : cus,
             causal ? 256 : 512);
}

int64_t rows_part(const sb::AttnArgs &a, const Plan &p) { // floats of the splits' rows
  return p.splits > 1 ? up(p.splits * a.B * a.Hk * a.rows * (int64_t)a.D, 4) : 0;
}
// (of dq in 16 bits beside its rows: their means, and two numbers of each)
int64_t rows_part_mean(const sb::AttnArgs &a, const Plan &p, int dtype) {
  return dtype == SB_F32 ? 0 : rows_part(a, p);
}
int64_t rows_part_left(const sb::AttnArgs &a, const Plan &p, int dtype) {
  return dtype == SB_F32 || p.splits == 1 ? 0 : up(2 * p.splits * a.B * a.Hk * (int64_t)a.rows, 4);
}
int64_t rows_part_lse(const sb::AttnArgs &a, const Plan &p) {
  return p.splits > 1 ? up(p.splits * a.B * a.Hk * (int64_t)a.rows, 4) : 0;
}
int64_t keys_part(const sb::AttnArgs &a, const Plan &p) {
  return p.splits > 1 ? up(2 * p.splits * a.B * a.Hk * (int64_t)a.Lk * a.D, 4) : 0;
}
int64_t delta_floats(const sb::AttnArgs &a) { return up((int64_t)a.B * a.Hk * a.rows, 4); }
int64_t peak_floats(const sb::AttnArgs &a, int dtype) {
  return dtype == SB_F16 ? up((int64_t)a.B * a.Hk * ((a.rows + 31) / 32), 4) : 0;
}

// (the workspace's size goes by the shape alone: the largest need)
int64_t forward_floats(const sb::AttnArgs &a, int dtype) {
  int64_t most = 0;
  for (const bool lengths : {false, true}) {
    const Plan p = plan_rows(a, dtype, true, false, lengths);
    most = std::max(most, rows_part(a, p) + rows_part_lse(a, p));
  }
  return most;
}
int64_t backward_floats(const sb::AttnArgs &a, int dtype) {
  int64_t most = 0;
  for (const bool causal : {false, true}) {
    most = std::max(most, keys_part(a, plan_keys(a, dtype, causal)));
    for (const bool lengths : {false, true}) {
      const Plan p = plan_rows(a, dtype, false, causal, lengths);
      most = std::max(most, rows_part(a, p) + rows_part_mean(a, p, dtype) + rows_part_left(a, p, dtype));
    }
  }
  return delta_floats(a) + peak_floats(a, dtype) + most;
}

int check_workspace(const void *workspace, size_t bytes, int64_t need) {
  if (need > 0 && (!workspace || !sb::aligned(workspace, 16)))
    return failf(SB_EARG, "workspace must be 16-byte aligned device memory");
  if (need > 0 && bytes < (size_t)need)
    return failf(SB_EWORKSPACE, "workspace too small: %zu bytes given, %lld needed", bytes, (long long)need);
  return SB_OK;
}

// launches of as many units as a grid takes: fewer than 2^24 blocks, and fewer than
// 2^32 threads (kMaxBlocksX counts 256 of them to a block)
template <class F> hipError_t over_units(sb::AttnArgs a, const Plan &p, F launch) {
  const int64_t grid = p.waves > sb::kAttnWaves ? sb::kMaxBlocksX / 2 : sb::kMaxBlocksX;
  a.tiles = (int32_t)p.tiles;
  a.splits = (int32_t)p.splits;
  a.span = (int32_t)p.span;
  a.div_set = sb::make_fastdiv((uint32_t)(8 * p.tiles * p.splits));
  a.div_splits = sb::make_fastdiv((uint32_t)p.splits);
  const int64_t units = (int64_t)a.B * a.Hk, each = p.tiles * p.splits, most = std::max<int64_t>(1, grid / each);
  for (int64_t u = 0; u < units; u += most) {
    a.unit0 = (uint32_t)u;
    a.units = (uint32_t)std::min(most, units - u);
    a.blocks = (uint32_t)(a.units * each);
    const hipError_t e = launch(a);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

int launched(hipError_t e) {
  return e == hipSuccess ? SB_OK : failf(SB_ELAUNCH, "attention launch failed: %s", hipGetErrorString(e));
}

} // namespace

extern "C" size_t attention_forward_workspace_bytes(const int64_t shape[6], int dtype) {
  sb::AttnArgs a;
  if (read_shape(shape, dtype, a)) return (size_t)-1;
  return (size_t)forward_floats(a, dtype) * sizeof(float);
}

extern "C" size_t attention_backward_workspace_bytes(const int64_t shape[6], int dtype) {
  sb::AttnArgs a;
  if (read_shape(shape, dtype, a)) return (size_t)-1;
  return (size_t)backward_floats(a, dtype) * sizeof(float);
}

extern "C" int attention_forward(const void *q, const int64_t q_stride[3], const void *k, const int64_t k_stride[3],
                                 const void *v, const int64_t v_stride[3], const int64_t shape[6], int dtype,
                                 float scale, int causal, const int32_t *query_lengths, const int32_t *key_lengths,
                                 void *out, const int64_t out_stride[3], float *lse, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  sb::AttnArgs a;
  int rc;
  if ((rc = read_shape(shape, dtype, a)) || (rc = check_scale(scale, a)) ||
      (rc = check_lengths(query_lengths, key_lengths, a)))
    return rc;
  if (!sb::aligned(lse, 4)) return failf(SB_EARG, "lse must be aligned to its element size");
  if (a.B == 0 || a.Lq == 0) return SB_OK;
  const int64_t Hq = (int64_t)a.Hk * a.group;
  Heads hq, hk, hv, ho;
  if ((rc = read_heads("q", q, q_stride, a, a.Lq, Hq, dtype, a.q, hq)) ||
      (rc = read_heads("k", k, k_stride, a, a.Lk, a.Hk, dtype, a.k, hk)) ||
      (rc = read_heads("v", v, v_stride, a, a.Lk, a.Hk, dtype, a.v, hv)) ||
      (rc = read_heads("out", out, out_stride, a, a.Lq, Hq, dtype, a.out, ho)) || (rc = check_distinct(ho)) ||
      (rc = check_apart(ho, hq, dtype)) || (rc = check_apart(ho, hk, dtype)) || (rc = check_apart(ho, hv, dtype)))
    return rc;
  if ((rc = check_workspace(workspace, workspace_bytes, forward_floats(a, dtype) * (int64_t)sizeof(float)))) return rc;
  a.causal = causal != 0;
  a.lse = lse;
  const Plan p = plan_rows(a, dtype, true, a.causal, a.q_len || a.k_len);
  const hipStream_t st = (hipStream_t)stream;
  // Causal tiles of which a CU holds two or more and a unit has one to two and a half
  // for each of its share of the CUs: the longest beside the shortest, and what is over,
  // the shortest of all, last.  16 heads in 4 groups of two samples fp32, against longest
  // first: 1280, 2080 and 2560 tokens of heads of 80 163, 274 and 393 us (172, 320 and
  // 412), of 32 58, 94 and 138 (63, 121 and 164), of 128 198, 328 and 490 (219, 415 and
  // 534); 16-bit heads of 40 to 192 the same either way.  Where a CU holds one tile, the
  // second ones do come second: heads of 160 fp32 285, 607 and 857 (285, 504 and 808), of
  // 256 bf16 84, 181 and 244 (84, 155 and 236).
  const int64_t units = (int64_t)a.B * a.Hk, beside = sb_cu_count() / units;
  if (a.causal && !a.q_len && !a.k_len && p.waves == sb::kAttnWaves && p.splits == 1 && units <= 8 &&
      p.tiles > beside && 2 * p.tiles <= 5 * beside &&
      sb::attn_forward_waves(sb::elem_bytes(dtype), sb::attn_padded(a.D), p.waves) > 1)
    a.beside = (int32_t)beside;
  if (p.splits > 1) {
    a.part = (float *)workspace;
    a.part_lse = a.part + rows_part(a, p);
  }
  hipError_t e = over_units(a, p, [&](const sb::AttnArgs &b) { return sb_launch_attention(b, dtype, p.waves, st); });
  if (e == hipSuccess && p.splits > 1) {
    a.splits = (int32_t)p.splits;
    e = sb_launch_attention_join(a, dtype, st);
  }
  return launched(e);
}

extern "C" int attention_backward(const void *dout, const int64_t dout_stride[3], const void *q,
                                  const int64_t q_stride[3], const void *k, const int64_t k_stride[3], const void *v,
                                  const int64_t v_stride[3], const void *out, const int64_t out_stride[3],
                                  const float *lse, const int64_t shape[6], int dtype, float scale, int causal,
                                  const int32_t *query_lengths, const int32_t *key_lengths, void *dq,
                                  const int64_t dq_stride[3], void *dk, const int64_t dk_stride[3], void *dv,
                                  const int64_t dv_stride[3], void *workspace, size_t workspace_bytes, void *stream) {
  sb::AttnArgs a;
  int rc;
  if ((rc = read_shape(shape, dtype, a)) || (rc = check_scale(scale, a)) ||
      (rc = check_lengths(query_lengths, key_lengths, a)))
    return rc;
  if (a.B == 0) return SB_OK;
  if (a.Lq > 0 && (!lse || !sb::aligned(lse, 4)))
    return failf(SB_EARG, "lse must be device memory aligned to its element size");
  const int64_t Hq = (int64_t)a.Hk * a.group;
  Heads in[5], to[3];
  if ((rc = read_heads("dout", dout, dout_stride, a, a.Lq, Hq, dtype, a.dout, in[0])) ||
      (rc = read_heads("q", q, q_stride, a, a.Lq, Hq, dtype, a.q, in[1])) ||
      (rc = read_heads("k", k, k_stride, a, a.Lk, a.Hk, dtype, a.k, in[2])) ||
      (rc = read_heads("v", v, v_stride, a, a.Lk, a.Hk, dtype, a.v, in[3])) ||
      (rc = read_heads("out", out, out_stride, a, a.Lq, Hq, dtype, a.out, in[4])) ||
      (rc = read_heads("dq", dq, dq_stride, a, a.Lq, Hq, dtype, a.dq, to[0])) ||
      (rc = read_heads("dk", dk, dk_stride, a, a.Lk, a.Hk, dtype, a.dk, to[1])) ||
      (rc = read_heads("dv", dv, dv_stride, a, a.Lk, a.Hk, dtype, a.dv, to[2])))
    return rc;
  for (int x = 0; x < 3; ++x) {
    if ((rc = check_distinct(to[x]))) return rc;
    for (int y = 0; y < 5; ++y)
      if ((rc = check_apart(to[x], in[y], dtype))) return rc;
    for (int y = 0; y < x; ++y)
      if ((rc = check_apart(to[x], to[y], dtype))) return rc;
  }
  if ((rc = check_workspace(workspace, workspace_bytes, backward_floats(a, dtype) * (int64_t)sizeof(float)))) return rc;
  a.causal = causal != 0;
  a.lse = const_cast<float *>(lse); // only read
  a.delta = (float *)workspace;
  a.peak = a.delta + delta_floats(a);
  float *const part = a.peak + peak_floats(a, dtype);
  const hipStream_t st = (hipStream_t)stream;
  hipError_t e = hipSuccess;
  if (a.Lq > 0) {
    const Plan p = plan_rows(a, dtype, false, a.causal, a.q_len || a.k_len);
    a.part = p.splits > 1 ? part : nullptr;
    a.part_mean = part + rows_part(a, p);
    a.part_left = a.part_mean + rows_part_mean(a, p, dtype);
    e = over_units(a, p, [&](const sb::AttnArgs &b) { return sb_launch_attention_dq(b, dtype, p.waves, whole_chunks(a, dtype), st); });
    a.splits = (int32_t)p.splits;
    if (e == hipSuccess && p.splits > 1)
      e = dtype == SB_F32 ? sb_launch_attention_sum(a, &a.dq, 1, a.rows, a.group, dtype, st)
                          : sb_launch_attention_dq_join(a, dtype, st);
  }
  if (e == hipSuccess && a.Lk > 0) {
    const Plan p = plan_keys(a, dtype, a.causal);
    a.part = p.splits > 1 ? part : nullptr;
    e = over_units(a, p, [&](const sb::AttnArgs &b) { return sb_launch_attention_dkv(b, dtype, whole_chunks(a, dtype), st); });
    a.splits = (int32_t)p.splits;
    const sb::AttnHeads to_[2] = {a.dk, a.dv};
    if (e == hipSuccess && p.splits > 1) e = sb_launch_attention_sum(a, to_, 2, a.Lk, 1, dtype, st);
  }
  return launched(e);
}
