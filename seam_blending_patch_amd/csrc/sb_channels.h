// sb_channels.h -- launch arguments of the channels-last group norm and of
// dropout, shared by the host entry points and the gfx950 kernels.
#pragma once

#include "sb_internal.h"

namespace sb {

// ---------------------------------------------------------------------------
// group norm, channels last
// ---------------------------------------------------------------------------
// x [N, S, C]: position (n, s) starts n * n stride + s * s stride elements from
// the base, C contiguous.
struct SampleStride {
  int64_t n, s;
};

constexpr int kChanThreads = 256; // of the blocks that go along the positions
constexpr int kMergeThreads = 1024;
// A group (or the few that fill whole vectors) that a block holds in registers needs
// one launch and is read once: vectors of a thread, forward and backward.
constexpr int kHeldThreads = 1024, kHeldVectors = 8, kHeldBackThreads = 512, kHeldBackVectors = 10;
constexpr int kChanBatch = 8;     // positions of a thread in flight

struct ChanArgs {
  const void *x, *dy;
  void *out; // y, or dx
  const void *gamma, *beta;
  void *dgamma, *dbeta;
  SampleStride sx, sdy, sout;
  int32_t N, S, C, G, Cg;
  int32_t NV, CV, RB;    // vectors of a position; of a block's columns; positions of a block at a time
  int32_t slabs;         // of CV vectors to a position
  int32_t chunks, chunk; // of a sample, positions of one
  int32_t apply_chunks, apply_chunk; // of the pass that writes, which leaves no partials
  uint32_t last;         // blocks go backwards from this one (0: forwards)
  int32_t silu;
  int32_t far;           // the output is more than the caches hold
  float eps;
  int32_t sg, CS;        // groups held by one block, channels of those (whole vectors); 0: the passes over blocks
  FastDiv div_CVs;       // vectors of those channels
  float *stats;          // [N][G][3]: the mean in two parts, 1 / sigma
  float *part;           // forward [N][chunks][3][C]: means in two parts, sums of squares about them;
                         // backward [N][chunks][2][C]: sums of g and of g h
  float *coef;           // [N][G][2] backward: the means of gamma g and of gamma g h
  FastDiv div_CV, div_Cg, div_slabs, div_chunks;
  uint32_t block0;       // of this launch
};

} // namespace sb

hipError_t sb_launch_channels_norm(const sb::ChanArgs &a, int dtype, int wdtype, hipStream_t st);
hipError_t sb_launch_channels_norm_backward(const sb::ChanArgs &a, int dtype, int wdtype, hipStream_t st);

namespace sb {

// ---------------------------------------------------------------------------
// dropout
// ---------------------------------------------------------------------------
constexpr int kDropThreads = 256;
constexpr int kDropVectors = 2; // of a thread

struct DropArgs {
  const void *x, *residual; // residual: nullptr, none
  void *out;
  int64_t sx[2], sr[2], so[2]; // {outer, inner} strides in elements
  FastDiv inner, div_units;
  int64_t D;                 // elements of a row
  int64_t row0;              // its row
  int64_t e0;                // its element of that row (launches that cut a row have only that)
  uint32_t units;            // 16-byte steps of this launch
  uint32_t threshold;        // words below it drop their element
  uint32_t site;
  float scale;
  const int64_t *state;      // {seed, offset}
  int32_t quads;             // rows begin at words that are multiples of 4
  int32_t far;               // the output is more than the caches hold
};

} // namespace sb

hipError_t sb_launch_dropout(const sb::DropArgs &a, int dtype, hipStream_t st);
