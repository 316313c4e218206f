// adapters.h -- what the launches of hb_adapters share: the plan's segments and
// a launch's parameters (adapters.cu: plan, checks and the short rows' kernels;
// adapters_long.cuh: the long tiles' kernels).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "hb_internal.h"
#include "ptx.cuh"

namespace hb {

constexpr int kAdShortRows = 16;        // rows of a short segment (at most)
constexpr int kAdTileRows = 128;        // rows of a long tile (at most)
constexpr int kAdMaxRank = 128;

struct AdapterSeg {
  int32_t adapter;      // -1: rows without one
  int32_t first;        // of the row list
  int32_t rows;
  int32_t token;        // long tiles: their first row; else -1
};

// When a launch waits for the one before it: before it reads anything; before
// it reads that launch's results (what was there before that launch is complete
// once it has let this one start); or at its end, needing nothing of it, so that
// its own completion stands for both.
enum AdapterWait : int32_t { kWaitFirst = 0, kWaitResults = 1, kWaitLast = 2 };

// One launch's segments and what it needs of the call.
struct AdapterParams {
  const AdapterSeg* segs;              // of this kind
  const int32_t* rows;                 // the row list
  int32_t num_segs, num_rows;          // of this kind
  int32_t first_row;                   // their first entry of the row list
  int32_t wait;                        // AdapterWait
  int32_t K, R, slices, N, ranks;      // ranks = slices * R
  const uint16_t *x, *a, *b;
  const int32_t* rank;
  const float* scale;
  int32_t pieces, units_per_piece;     // of K, in units of 64
  int32_t groups;                      // of ranks
  const uint16_t* y[3];
  uint16_t* out[3];
  int32_t cols[3];
  int32_t chunks[3], chunk_cols;       // column chunks (long: 128-column blocks) per destination
  // short
  float* h;                            // [pieces, num_rows, ranks]
  int32_t group_ranks;
  // long
  uint16_t* terms;                     // [2 terms, num_segs * 128, h_cols] of h, scale included
  int32_t h_cols, h_slice;             // h_slice: a destination's ranks, whole steps of 16
  int32_t boxes;                       // 16-rank boxes of a shrink CTA (at most)
  int* dev_error;
};

// ranks read as if held to [0, R]
__device__ __forceinline__ int rank_of(const AdapterParams& p, int adapter) {
  return adapter < 0 ? 0 : min(max(__ldg(p.rank + adapter), 0), p.R);
}

// a and b as bf16 pairs hi + lo (what is not finite is hi alone)
__device__ __forceinline__ void two_terms(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  const float ra = a - bf16lo_to_f32(hi), rb = b - bf16hi_to_f32(hi);
  lo = pack_bf16x2(isfinite(ra) ? ra : 0.f, isfinite(rb) ? rb : 0.f);
}

}  // namespace hb
