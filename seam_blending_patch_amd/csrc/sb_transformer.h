// sb_transformer.h -- launch arguments shared by the host entry points and the
// gfx950 kernels of the transformer operators (layer norm, rotary embedding,
// gradient norm and clipping).
#pragma once

#include "sb_internal.h"

namespace sb {

constexpr int64_t kLastLevelBytes = (int64_t)256 << 20; // the memory-side cache

// ---------------------------------------------------------------------------
// layer norm
// ---------------------------------------------------------------------------
// Rows are indexed r = o * inner + i; a tensor's row r starts o * outer stride
// + i * inner stride elements from its base.
struct RowStride {
  int64_t o, i;
};

struct LNArgs {
  const void *x, *dy;
  void *out; // y, or dx
  const void *gamma, *beta;
  RowStride sx, sdy, sout;
  int64_t rows;
  FastDiv inner;
  int32_t D;
  float eps, inv_d;
  int32_t far;        // the output is more than the caches hold
  // rows split into chunks
  float *rowstat;     // 8 floats a row: K, E, 1/sigma, mean of g, mean of g h
  float *chunks;      // 8 floats a chunk of a row
  // backward
  float *part;        // weight-gradient partials [blocks][2][columns] (nullptr: none wanted)
  void *dgamma, *dbeta;
  int32_t nparts, cols; // blocks (of partials); floats of each (the columns, rounded up to the block's)
};

constexpr int kLNThreads = 256; // threads of a block of rows, of a chunk or of columns
// rows of more vectors are split: forward, and (backward_layout) backward
constexpr int64_t kForwardVectors = 4096, kBackwardVectors = 2048;
constexpr int kChunkVectors = 4; // vectors of a chunk on each of kLNThreads threads

// How the backward pass lays rows of nv 16-byte vectors over threads: NV
// vectors on each of LANES threads, as many rows to a block as it has room for
// (lanes 0: the row is too long for registers and is split into chunks).
// A wave to a row as long as the sums of its columns fit its registers: it
// needs no barrier; then the fewest waves.  Measured in us, kernel and reduction
// (copy rate: 156 us for each of these but the last, 37):
//   65536 x 2048 fp16:   64 x 4 157 (1, 3, 4 blocks a CU 175, 163, 158)
//   32768 x 4096 bf16:  128 x 4 156
//   16384 x 8192 bf16:  256 x 4 171   512 x 2 209
//   8192 x 16384 bf16: 1024 x 2 183   512 x 4 178 (fp32, twice the bytes: 298, 313)
//   243360 x 128 bf16:   16 x 1 41 (3, 6, 8 blocks a CU 43, 41, 44)
struct LNLayout {
  int lanes, nv;
  int threads() const { return lanes > kLNThreads ? lanes : kLNThreads; }
  int rows() const { return threads() / lanes; } // of a block, at a time
  // few blocks: each adds a row of partials to be written and read again; more
  // of them only where a thread has little in flight
  int blocks_per_cu() const { return nv == 1 ? 4 : lanes > kLNThreads ? 1 : 2; }
};
inline LNLayout backward_layout(int64_t nv) {
  if (nv <= 64) {
    int lanes = 4;
    while (lanes < nv) lanes *= 2;
    return LNLayout{lanes, 1};
  }
  if (nv <= 256) return LNLayout{64, (int)(nv + 63) / 64};
  if (nv <= 512) return LNLayout{128, nv <= 384 ? 3 : 4};
  if (nv <= 1024) return LNLayout{256, nv <= 768 ? 3 : 4};
  if (nv <= kBackwardVectors) return LNLayout{1024, 2};
  return LNLayout{0, 0};
}

// ---------------------------------------------------------------------------
// rotary position embedding
// ---------------------------------------------------------------------------
constexpr int kRotaryMaxAxes = 4;
constexpr int kRotaryThreads = 256;

struct RotaryTensor {
  const void *in;
  void *out;
  int64_t in_b, in_t, in_h, out_b, out_t, out_h; // strides in elements
};

struct RotaryArgs {
  RotaryTensor x[2];     // query heads, key heads
  int32_t heads[2];
  uint32_t token0, tokens; // of this launch, of all batch * length
  FastDiv length;
  int32_t D, part;       // head length, rotated elements (even)
  int32_t units_turned, units; // 16-byte steps of a head: over its pairs, and with those over the rest
  int32_t items;         // steps of a token (all its heads)
  FastDiv div_units, div_items, div_half;
  const double *freqs;   // radians per position, part / 2 of them
  const void *positions;
  int64_t pos_axis, pos_b, pos_t; // strides in elements
  int32_t pos64;         // positions are int64 (else int32)
  int32_t axes, ends[kRotaryMaxAxes]; // pairs [ends[a - 1], ends[a]) turn by the positions of axis a
  float scale, scale_sin;  // cosines and sines are multiplied by these (the sign of the direction in the second)
};

// ---------------------------------------------------------------------------
// gradient norm and clipping
// ---------------------------------------------------------------------------
constexpr int kClipTensors = 128; // tensors of a launch (their table is a kernel argument)
constexpr int kClipThreads = 256;

struct ClipArgs {
  const void *in[kClipTensors];
  void *out[kClipTensors];
  int64_t n[kClipTensors];
  uint32_t begin[kClipTensors + 1]; // first chunk of each tensor
  uint8_t types[kClipTensors];      // dtype, and dtype of the output << 2
  int64_t chunk;                    // elements of a chunk (a multiple of kClipThreads vectors)
  double *partials;                 // sums of squares: this launch's first, or all of them (second pass)
  int32_t tensors, npartials, nt;   // nt: store the outputs past the caches
  float max_norm, eps;
  float *norm;                      // written by the first block of a second-pass launch that has it
};
static_assert(sizeof(ClipArgs) <= 4096, "kernel arguments of at most 4 KiB");

} // namespace sb

hipError_t sb_launch_layer_norm(const sb::LNArgs &a, int dtype, int wdtype, hipStream_t st);
hipError_t sb_launch_layer_norm_backward(const sb::LNArgs &a, int dtype, int wdtype, hipStream_t st);
hipError_t sb_launch_rotary(const sb::RotaryArgs &a, int dtype, int interleaved, hipStream_t st);
hipError_t sb_launch_square_sums(const sb::ClipArgs &a, unsigned blocks, hipStream_t st);
hipError_t sb_launch_clip(const sb::ClipArgs &a, unsigned blocks, hipStream_t st);
