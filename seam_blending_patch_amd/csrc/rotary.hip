// rotary.hip -- rotary position embedding of query and key heads, gfx950.
//
// Pair i of a head at token t is turned by the angle a = p f_i, p the token's
// position on the pair's axis:
//   (u, v) -> scale (u cos a - v sin a, u sin a + v cos a);
// pairs are neighbours (interleaved) or half the rotated part apart.  The
// transpose (the gradient) turns by -a.
//
// The angle is formed in 64 bits as turns and reduced by its nearest whole
// number before it is rounded to fp32, so that a position of a million costs
// no accuracy; cosine and sine are then fp32 functions of at most half a turn.

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
  float s, c;
  sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
  return make_float2(c * A.scale, s * A.scale_sin);
}

// One block a token; a thread takes 16-byte steps of its heads (half layout:
// a step of each half).
template <int DT, bool INTER>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(const RotaryArgs A) {
  constexpr int V = kVec<DT>;
  const int half = A.part / 2, items = (A.heads[0] + A.heads[1]) * A.units;
  for (int64_t token = blockIdx.x; token < A.tokens; token += gridDim.x) {
    const uint32_t b = fdiv((uint32_t)token, A.length), t = (uint32_t)token - b * A.length.d;
    for (int item = threadIdx.x; item < items; item += kRotaryThreads) {
      const int head = fdiv(item, A.div_units), unit = item - head * A.units;
      const bool key = head >= A.heads[0];
      const RotaryTensor &T = A.x[key];
      const int h = key ? head - A.heads[0] : head;
      const int64_t in = b * T.in_b + t * T.in_t + h * T.in_h, out = b * T.out_b + t * T.out_t + h * T.out_h;
      if (unit >= A.units_turned) {
        const int e = A.part + (unit - A.units_turned) * V;
        if (T.in != T.out) store_part<DT>(T.out, out + e, A.D - e, load_part<DT>(T.in, in + e, A.D - e));
        continue;
      }
      if constexpr (INTER) {
        const int e = unit * V;
        float f[V];
        unpack<DT, 16>(load_part<DT>(T.in, in + e, A.part - e), f);
#pragma unroll
        for (int k = 0; k < V; k += 2) {
          if (e + k >= A.part) break;
          const float2 cs = cos_sin(A, (e + k) >> 1, b, t);
          const float u = f[k], v = f[k + 1];
          f[k] = fmaf(u, cs.x, -(v * cs.y));
          f[k + 1] = fmaf(u, cs.y, v * cs.x);
        }
        store_part<DT>(T.out, out + e, A.part - e, pack<DT, 16>(f));
      } else {
        const int e = unit * V, n = half - e;
        float u[V], v[V];
        unpack<DT, 16>(load_part<DT>(T.in, in + e, n), u);
        unpack<DT, 16>(load_part<DT>(T.in, in + half + e, n), v);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          if (k >= n) break;
          const float2 cs = cos_sin(A, e + k, b, t);
          const float a = u[k];
          u[k] = fmaf(a, cs.x, -(v[k] * cs.y));
          v[k] = fmaf(a, cs.y, v[k] * cs.x);
        }
        store_part<DT>(T.out, out + e, n, pack<DT, 16>(u));
        store_part<DT>(T.out, out + half + e, n, pack<DT, 16>(v));
      }
    }
  }
}

template <int DT, bool INTER> hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st) {
  const unsigned blocks = (unsigned)std::min<int64_t>(a.tokens, kMaxBlocksX);
  hipLaunchKernelGGL((rotary_kernel<DT, INTER>), dim3(blocks), dim3(kRotaryThreads), 0, st, a);
  return hipGetLastError();
}

} // namespace sb

hipError_t sb_launch_rotary(const sb::RotaryArgs &a, int dtype, int interleaved, hipStream_t st) {
  using namespace sb;
  if (dtype == DT_F32) return interleaved ? launch_rotary<DT_F32, true>(a, st) : launch_rotary<DT_F32, false>(a, st);
  if (dtype == DT_F16) return interleaved ? launch_rotary<DT_F16, true>(a, st) : launch_rotary<DT_F16, false>(a, st);
  return interleaved ? launch_rotary<DT_BF16, true>(a, st) : launch_rotary<DT_BF16, false>(a, st);
}
