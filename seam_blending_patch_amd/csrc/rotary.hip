// rotary.hip -- rotary position embedding of query and key heads, gfx950.
//
// Pair i of a head at token t is turned by the angle a = p f_i, p the token's
// position on the pair's axis:
//   (u, v) -> scale (u cos a - v sin a, u sin a + v cos a);
// pairs are neighbours (interleaved) or half the rotated part apart.  The
// transpose (the gradient) turns by -a.
//
// The angle is formed in 64 bits as turns and reduced by its nearest whole
// number, so that a position of a million costs no accuracy; cosine and sine are
// then fp32 functions of at most half a turn, rounded to fp32, and the little
// that this rounding left out (up to 2^-26 turns, more than an fp32 cosine's own
// error) turns them on by its own first order.

#include "sb_row.h"
#include "sb_transformer.h"

#include <algorithm>

namespace sb {

__device__ __forceinline__ int64_t read_position(const RotaryArgs &A, int axis, uint32_t b, uint32_t t) {
  const int64_t i = axis * A.pos_axis + b * A.pos_b + t * A.pos_t;
  return A.pos64 ? ((const int64_t *)A.positions)[i] : (int64_t)((const int32_t *)A.positions)[i];
}

__device__ __forceinline__ float2 cos_sin(const RotaryArgs &A, int pair, uint32_t b, uint32_t t) {
  int axis = 0;
#pragma unroll
  for (int a = 0; a + 1 < kRotaryMaxAxes; ++a) axis += a + 1 < A.axes && pair >= A.ends[a];
  constexpr double kTurns = 0.15915494309189533577; // 1 / (2 pi)
  const double turns = (double)read_position(A, axis, b, t) * (A.freqs[pair] * kTurns);
  const double part = turns - rint(turns);
  const float near = (float)part, rest = 6.28318531f * (float)(part - (double)near);
  float s, c;
  sincospif(2.0f * near, &s, &c);
  return make_float2(fmaf(-s, rest, c) * A.scale, fmaf(c, rest, s) * A.scale_sin);
}

// field by field, so that it is selects among scalar registers and no load at
// an address that differs from lane to lane
__device__ __forceinline__ RotaryTensor tensor_of(const RotaryArgs &A, bool key) {
  const RotaryTensor &q = A.x[0], &k = A.x[1];
  return RotaryTensor{key ? k.in : q.in,     key ? k.out : q.out,     key ? k.in_b : q.in_b,  key ? k.in_t : q.in_t,
                      key ? k.in_h : q.in_h, key ? k.out_b : q.out_b, key ? k.out_t : q.out_t, key ? k.out_h : q.out_h};
}

// A thread takes one 16-byte step of a head (in the half layout one of each
// half), a block the next 256 of all tokens', wherever tokens begin and end, so
// that no thread is idle.  The cosines and sines of the tokens it touches are
// formed once, by all its threads, and kept in LDS for every head; the step is
// requested before that.
//
// Bound by the copy of the heads: 20280 tokens of 24 x 128 bf16, interleaved,
// 250 MB in 46.5 to 51 us (4.9 to 5.4 TB/s, the rate of a large copy), 16384
// tokens of 40 x 128 in halves 335 MB in 58 to 62 us.  Measured against it:
// whole tokens to a block 61 us for the first of these (a third of the threads
// idle), an angle for every head's step of its own 109 us; 2 and 4 steps a
// thread 44.3 and 46.2 us for the first but 62 and 67 us for the second.  With
// one head to a key, 64 pairs of angles to every 256 bytes, the angles show:
// 65536 tokens, 67 MB, in 19.8 us (3.4 TB/s; 19.4 if their rounding stayed).
template <int DT, bool INTER>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(const RotaryArgs A) {
  constexpr int V = kVec<DT>;
  extern __shared__ float2 turn[]; // [tokens of the block][pairs]
  const int half = A.part / 2;
  const uint32_t total = A.tokens * A.items; // below 2^31
  const uint32_t base = blockIdx.x * kRotaryThreads, item = base + threadIdx.x;
  const uint32_t row0 = fdiv(base, A.div_items), row = fdiv(item, A.div_items);
  const uint32_t j = item - row * A.items, head = fdiv(j, A.div_units), unit = j - head * A.units;
  const bool key = head >= (uint32_t)A.heads[0], turned = unit < (uint32_t)A.units_turned;
  const RotaryTensor T = tensor_of(A, key);
  const int e = turned ? unit * V : A.part + (unit - A.units_turned) * V;
  int64_t out = 0;
  int count = 0; // elements to read and write (no more than a vector of them)
  Vec<16> first, second;
  if (item < total) {
    const uint32_t b = fdiv(A.token0 + row, A.length), t = A.token0 + row - b * A.length.d;
    const uint32_t h = key ? head - A.heads[0] : head;
    const int64_t in = b * T.in_b + t * T.in_t + h * T.in_h;
    out = b * T.out_b + t * T.out_t + h * T.out_h + e;
    if (turned) count = (INTER ? A.part : half) - e;
    else if (T.in != T.out) count = A.D - e; // what is not turned stays where it is in place
    // whole vectors of the head, also where fewer elements are the step's own;
    // where the head ends, moved into place below
    if (count > 0) first = request_row<DT, CUT>(T.in, in, e, A.D);
    if (!INTER && turned) second = request_row<DT, CUT>(T.in, in, half + e, A.D);
  }
  const uint32_t rows = fdiv(min(base + kRotaryThreads, total) - 1, A.div_items) + 1 - row0;
  for (uint32_t i = threadIdx.x; i < rows * half; i += kRotaryThreads) {
    const uint32_t r = fdiv(i, A.div_half), token = A.token0 + row0 + r, b = fdiv(token, A.length);
    turn[i] = cos_sin(A, i - r * half, b, token - b * A.length.d);
  }
  __syncthreads();
  if (count <= 0) return;
  settle_row<DT, CUT>(first, e, A.D);
  if (turned) {
    float u[V], v[V];
    unpack<DT, 16>(first, u);
    if constexpr (INTER) {
      const float2 *cs = turn + (row - row0) * half + e / 2;
#pragma unroll
      for (int k = 0; k < V; k += 2)
        if (k < count) {
          const float2 c = cs[k / 2];
          const float a = u[k];
          u[k] = fmaf(a, c.x, -(u[k + 1] * c.y));
          u[k + 1] = fmaf(a, c.y, u[k + 1] * c.x);
        }
    } else {
      const float2 *cs = turn + (row - row0) * half + e;
      settle_row<DT, CUT>(second, half + e, A.D);
      unpack<DT, 16>(second, v);
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (k < count) {
          const float2 c = cs[k];
          const float a = u[k];
          u[k] = fmaf(a, c.x, -(v[k] * c.y));
          v[k] = fmaf(a, c.y, v[k] * c.x);
        }
      store_part<DT>(T.out, out + half, count, pack<DT, 16>(v));
    }
    first = pack<DT, 16>(u);
  }
  store_part<DT>(T.out, out, count, first);
}

template <int DT, bool INTER> hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st) {
  const int64_t total = a.tokens * (int64_t)a.items;
  // tokens that a block can touch; a token has at least half / V steps, so
  // their angles are at most 64 KiB (for heads of up to 2^13 elements)
  const int64_t rows = std::min<int64_t>((a.items - 1 + kRotaryThreads - 1) / a.items + 1, a.tokens);
  hipLaunchKernelGGL((rotary_kernel<DT, INTER>), dim3((unsigned)((total + kRotaryThreads - 1) / kRotaryThreads)),
                     dim3(kRotaryThreads), rows * (a.part / 2) * sizeof(float2), st, a);
  return hipGetLastError();
}

} // namespace sb

hipError_t sb_launch_rotary(const sb::RotaryArgs &a, int dtype, int interleaved, hipStream_t st) {
  using namespace sb;
  if (dtype == DT_F32) return interleaved ? launch_rotary<DT_F32, true>(a, st) : launch_rotary<DT_F32, false>(a, st);
  if (dtype == DT_F16) return interleaved ? launch_rotary<DT_F16, true>(a, st) : launch_rotary<DT_F16, false>(a, st);
  return interleaved ? launch_rotary<DT_BF16, true>(a, st) : launch_rotary<DT_BF16, false>(a, st);
}
