// dropout.hip -- dropout from a counter-based generator for gfx950.  The mask is
// never stored: element i takes word i % 4 of the generator at counter i / 4,
// forward and backward alike.
//
// Generator: Philox4x32 with ten rounds (Salmon, Moraes, Dror & Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011), 32 bits to an element.  Its 20 wide
// products to 4 elements hide behind the memory's time: 65536 x 2048 bf16 with a
// residual 139 us, 5.8 TB/s.
#include "sb_channels.h"
#include "sb_row.h"

namespace sb {
namespace {

struct Words {
  uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint32_t block, uint32_t site, uint64_t offset, uint64_t seed) {
  uint32_t a = block, b = site, c = (uint32_t)offset, d = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)0xD2511F53u * a, q = (uint64_t)0xCD9E8D57u * c;
    a = (uint32_t)(q >> 32) ^ b ^ k0;
    b = (uint32_t)q;
    c = (uint32_t)(p >> 32) ^ d ^ k1;
    d = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Words{{a, b, c, d}};
}

// QUADS: every vector begins at a multiple of 4 words; else its words come from
// one block more and are moved into place.
template <int DT, bool QUADS, bool RESIDUAL, bool FAR>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(const DropArgs a) {
  constexpr int V = kVec<DT>, U = kDropVectors, B = V / 4 + (QUADS ? 0 : 1);
  Vec<16> x[U], res[U];
  int64_t to[U];
  uint32_t block[U], shift[U];
  int n[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const uint32_t id = (blockIdx.x * U + j) * kDropThreads + threadIdx.x;
    n[j] = 0;
    if (id >= a.units) continue;
    const uint32_t row = fdiv(id, a.div_units);
    const int64_t e = a.e0 + (int64_t)(id - row * a.div_units.d) * V, r = a.row0 + row;
    const uint32_t o = fdiv((uint32_t)r, a.inner), i = (uint32_t)r - o * a.inner.d;
    n[j] = (int)min((int64_t)V, a.D - e);
    x[j] = load_part<DT>(a.x, o * a.sx[0] + i * a.sx[1] + e, n[j]);
    if (RESIDUAL) res[j] = load_part<DT>(a.residual, o * a.sr[0] + i * a.sr[1] + e, n[j]);
    to[j] = o * a.so[0] + i * a.so[1] + e;
    const uint64_t word = (uint64_t)(r * a.D + e);
    block[j] = (uint32_t)(word >> 2);
    shift[j] = (uint32_t)word & 3;
  }
  const uint64_t seed = (uint64_t)a.state[0], offset = (uint64_t)a.state[1];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    if (n[j] <= 0) continue;
    uint32_t w[4 * B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const Words p = philox(block[j] + b, a.site, offset, seed);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[4 * b + k] = p.w[k];
    }
    float f[V], r[V];
    unpack<DT, 16>(x[j], f);
    if (RESIDUAL) unpack<DT, 16>(res[j], r);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      uint32_t word = w[k];
      if constexpr (!QUADS) {
        word = pick(shift[j] & 1, w[k + 1], word);
        if (shift[j] & 2) word = pick(shift[j] & 1, w[k + 3], w[k + 2]);
      }
      const bool keep = word >= a.threshold;
      if (RESIDUAL) f[k] = keep ? __builtin_fmaf(f[k], a.scale, r[k]) : r[k];
      else f[k] = keep ? f[k] * a.scale : 0.0f;
    }
    store_part<DT, FAR>(a.out, to[j], n[j], pack<DT, 16>(f));
  }
}

template <int DT, bool QUADS> void launch(const DropArgs &a, dim3 grid, hipStream_t st) {
  const dim3 block(kDropThreads);
  if (a.residual) {
    if (a.far) hipLaunchKernelGGL((dropout_kernel<DT, QUADS, true, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((dropout_kernel<DT, QUADS, true, false>), grid, block, 0, st, a);
  } else if (a.far) {
    hipLaunchKernelGGL((dropout_kernel<DT, QUADS, false, true>), grid, block, 0, st, a);
  } else {
    hipLaunchKernelGGL((dropout_kernel<DT, QUADS, false, false>), grid, block, 0, st, a);
  }
}
template <int DT> hipError_t launch(const DropArgs &a, hipStream_t st) {
  const unsigned per = kDropThreads * kDropVectors;
  const dim3 grid((a.units + per - 1) / per);
  if (a.quads) launch<DT, true>(a, grid, st);
  else launch<DT, false>(a, grid, st);
  return hipGetLastError();
}

} // namespace
} // namespace sb

hipError_t sb_launch_dropout(const sb::DropArgs &a, int dtype, hipStream_t st) {
  if (dtype == sb::DT_F32) return sb::launch<sb::DT_F32>(a, st);
  if (dtype == sb::DT_F16) return sb::launch<sb::DT_F16>(a, st);
  return sb::launch<sb::DT_BF16>(a, st);
}
