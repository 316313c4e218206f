// adapters_long.cuh -- hb_adapters for long tiles (up to 128 rows that are
// neighbours in the batch: prompts) on the tcgen05 tensor cores: h = scale x A^T
// (shrink) and out = y + h B^T (expand).
//
// Every wait is bounded; a CTA allocates tensor memory only after its wait for
// the grid before it, so that no CTA holds it while waiting for another grid.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "adapters.h"
#include "hb_internal.h"
#include "ptx.cuh"

namespace hb {

// ---------------------------------------------------------------- shrink
// A cluster of CTAs takes a tile of rows and up to 192 ranks (16 at a time, those
// in use, of all destinations).  Each CTA sums a piece of K: the x tile and the
// adapter's ranks come by TMA into a ring of 64-wide K blocks, M 128, N the ranks,
// fp32 in tensor memory.  The pieces meet through distributed shared memory: each
// CTA adds up some of the ranks, in the order of the pieces, and writes their two
// bf16 terms where the expand launch reads them by TMA.
//
// Measured: 6005 rows of K 7168, ranks up to 64 of three destinations, 43 us for 121
// MB (100 CTAs in clusters of two).  A 64-wide K block takes 0.54 us with 9 boxes of
// ranks, 0.39 with 4: the TMA unit takes the x rows and the ranks, 128 bytes a row, at
// about 2.5 clocks each, and a CTA's start, exchange and end cost 9 us.  A ring of 104,
// 160 or 200 KB and one to five pieces are within 3 % of one another (only one CTA
// that uses tensor memory fits an SM); the ring of 104 KB leaves room for the short
// rows' CTAs.
constexpr int kLsThreads = 192;               // warp 0 TMA, warp 1 MMA, warps 2-5 epilogue
constexpr int kLsXBytes = kAdTileRows * 128;  // a 64-wide K block of the x tile
constexpr int kLsBoxBytes = 16 * 128;         // and of 16 ranks
constexpr int kLsMaxBoxes = 12;               // N 192 (at most)
constexpr int kLsMaxStages = 6;
constexpr int kLsMaxPieces = 16;              // CTAs of a cluster (at most; more than 8 only where they fit)
constexpr int kLsRingBytes = 104 * 1024;
constexpr int kLsBarBytes = (2 * kLsMaxStages + 1) * 8 + 24;
constexpr size_t kLsSmem = kLsRingBytes + kLsBarBytes + 1024;
static_assert(kLsMaxBoxes * 16 * kAdTileRows * 4 <= kLsRingBytes, "the sums fit the ring");
static_assert(2 * (kLsXBytes + kLsMaxBoxes * kLsBoxBytes) <= kLsRingBytes, "two stages at least");
static_assert(kLsSmem <= 227 * 1024, "shrink smem");

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

__global__ void __launch_bounds__(kLsThreads, 1)
    shrink_long_kernel(const AdapterParams p, const __grid_constant__ CUtensorMap xmap,
                       const __grid_constant__ CUtensorMap amap) {
  extern __shared__ uint8_t s_raw[];
  griddep_wait();
  griddep_launch_dependents();
  const int piece = blockIdx.x % p.pieces;              // = rank in the cluster
  const int at = blockIdx.x / p.pieces;
  const int tile = at % p.num_segs, group = at / p.num_segs;
  const AdapterSeg seg = p.segs[tile];
  const int rank = rank_of(p, seg.adapter);
  const int per_slice = (rank + 15) / 16;
  const int box0 = group * p.boxes, boxes = min(per_slice * p.slices - box0, p.boxes);
  if (boxes <= 0) return;                               // (the whole cluster)
  uint8_t* smem = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);
  const int stage_bytes = kLsXBytes + boxes * kLsBoxBytes, stages = min(kLsMaxStages, kLsRingBytes / stage_bytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kLsRingBytes);
  uint64_t* empty = full + kLsMaxStages;
  uint64_t* done = empty + kLsMaxStages;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  int* abort_i = reinterpret_cast<int*>(tmem_holder + 2);
  volatile int* abort_flag = abort_i;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float scale = __ldg(p.scale + seg.adapter);
  uint32_t tmem_cols = 32;
  while (tmem_cols < (uint32_t)boxes * 16u) tmem_cols *= 2;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_i = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;
  const int units = (p.K + 63) / 64;
  const int u0 = piece * p.units_per_piece, n = min(units, u0 + p.units_per_piece) - u0;   // (at least one)
  if (warp == 0) {
    // lane j brings box j of the ranks, lane 31 the rows of x
    const int b = box0 + min(lane, boxes - 1);
    const int a_row = (seg.adapter * p.slices + b / per_slice) * p.R + b % per_slice * 16;
    if (lane == 0) {
      tma_prefetch_desc(&xmap);
      tma_prefetch_desc(&amap);
    }
    fence_proxy_async_global();
    int i = 0;
    for (; i < n; ++i) {
      const int s = i % stages;
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ((i / stages) & 1) ^ 1, abort_flag))) break;
      uint8_t* st = smem + s * stage_bytes;
      if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(kLsXBytes + boxes * kLsBoxBytes));
      __syncwarp();
      if (lane == 31) tma_load_2d(st, &xmap, &full[s], (u0 + i) * 64, seg.token);
      else if (lane < boxes) tma_load_2d(st + kLsXBytes + lane * kLsBoxBytes, &amap, &full[s], (u0 + i) * 64, a_row);
      __syncwarp();
    }
    // before the ring is used again or the CTA exits, what was issued has landed
    for (int s = 0; s < stages && s < i; ++s) drain_wait(&full[s], ((i - 1 - s) / stages) & 1, abort_flag);
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(kAdTileRows, (uint32_t)boxes * 16u, false);
      for (int i = 0; i < n; ++i) {
        const int s = i % stages;
        if (!mbar_wait(&full[s], (i / stages) & 1, abort_flag)) break;
        tc_fence_after_sync();
        const uint32_t a = smem_u32(smem + s * stage_bytes), b = a + kLsXBytes;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_bf16(tmem, sdesc_sw128(a + kk * 32, 16, 1024), sdesc_sw128(b + kk * 32, 16, 1024), idesc,
                      (i > 0 || kk > 0) ? 1u : 0u);
        tc_commit(&empty[s]);
      }
      // every MMA issued completes before the accumulator is read or freed
      tc_commit(done);
      drain_wait(done, 0u, abort_flag);
    }
  } else {
    // this piece's sums, [rank][row], over the ring (all of it was consumed)
    const int row = (warp & 3) * 32 + lane;
    const bool got = __all_sync(0xffffffffu, mbar_wait(done, 0u, abort_flag) && !*abort_flag);
    tc_fence_after_sync();
    float* sums = reinterpret_cast<float*>(smem);
    for (int j = 0; got && j < boxes; j += 2) {
      uint32_t v[32];
      tmem_ld32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)j * 16u, v);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (j * 16 + e < boxes * 16) sums[(j * 16 + e) * kAdTileRows + row] = __uint_as_float(v[e]);
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  cluster_sync_all();
  if (warp >= 2) {
    const int row = (warp & 3) * 32 + lane;
    const uint32_t mine = smem_u32(smem) + (uint32_t)row * 4u;
    // eight ranks at a time, in turn among the CTAs; a thread has a row's eight
    for (int j = piece; j < 2 * boxes; j += p.pieces) {
      const uint32_t at_j = (uint32_t)(j * 8 * kAdTileRows) * 4u;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
      // (eight pieces' loads on their way at a time)
      for (int q0 = 0; q0 < p.pieces; q0 += 8) {
        float o[8][8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t src = mapa_shared(mine, (uint32_t)min(q0 + q, p.pieces - 1)) + at_j;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            o[q][e] = q0 + q < p.pieces ? ld_cluster_f32(src + (uint32_t)(e * kAdTileRows) * 4u) : 0.f;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += o[q][e];
      }
      const int b = box0 + (j >> 1), r0 = b % per_slice * 16 + (j & 1) * 8;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)   // (a rank that the adapter does not have may have met an infinity of x)
        two_terms(r0 + 2 * e < rank ? v[2 * e] * scale : 0.f, r0 + 2 * e + 1 < rank ? v[2 * e + 1] * scale : 0.f,
                  hi[e], lo[e]);
      uint16_t* dst = p.terms + ((int64_t)tile * kAdTileRows + row) * p.h_cols + b / per_slice * p.h_slice + r0;
      *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      dst += (int64_t)p.num_segs * kAdTileRows * p.h_cols;
      *reinterpret_cast<uint4*>(dst) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  __syncwarp();
  // no CTA leaves while another one may read its sums
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, tmem_cols);
  }
  if (threadIdx.x == 0 && *abort_flag) report_error(p.dev_error, HB_DEVERR_TIMEOUT);
}

// ---------------------------------------------------------------- expand
// Persistent: the blocks (128 rows of a tile, 128 columns of a destination) of
// all tiles stand in one row, tile after tile, and each CTA takes an equal share
// of them.  Warp 0 brings a block's y and rows of B (and, where a tile or a
// destination begins, the two terms of h) by TMA; warp 1 multiplies (tcgen05,
// M 128, N 128, two terms; accumulators of two blocks in tensor memory); warps
// 2-9 (thread = row, four warps to each half of the columns) add y to the sums in
// shared memory and write the rows out from there, 128 bytes at a time, only those
// of the tile.
//
// Measured: 6005 rows of N 9216 48.5 us for 221 MB of y (4.6 TB/s, 68 % of the copy
// rate; on warp MMAs 112 us); with four epilogue warps 54 us.
constexpr int kLeThreads = 320;
constexpr int kLeEpilogueWarps = 8;
constexpr int kLeCols = 128;                            // columns of a block
constexpr int kLePanel = 128 * 128;                     // bytes: 128 rows of 64 bf16 columns
constexpr int kLeMaxStages = 4;
constexpr int kLeBytes = 224 * 1024;                    // h and the ring
constexpr int kLeBarBytes = (2 * kLeMaxStages + 4 + 4 + 1) * 8 + 24;
constexpr size_t kLeSmem = kLeBytes + kLeBarBytes + 1024;
static_assert(kLeSmem <= 227 * 1024, "expand smem");

struct LeCfg {
  int panels;    // 64-rank panels of a term, and of a block's rows of B
  int hbufs;     // h of so many (tile, destination) pairs at a time
  int stages;
};
inline LeCfg le_cfg(int R) {
  LeCfg c;
  c.panels = (R + 63) / 64;
  c.hbufs = c.panels == 1 ? 2 : 1;
  c.stages = std::min(kLeMaxStages, (kLeBytes - c.hbufs * 2 * c.panels * kLePanel) / ((c.panels + 2) * kLePanel));
  return c;
}

struct LeMaps {
  CUtensorMap h, b, y[3];
};

// Where block i of the launch stands.
struct LeBlock {
  int tile, slice, col;    // col: first column in its destination
};
__device__ __forceinline__ LeBlock le_block(const AdapterParams& p, int i) {
  const int per_tile = p.chunks[0] + p.chunks[1] + p.chunks[2];
  LeBlock b;
  b.tile = i / per_tile;
  b.slice = 0;
  b.col = i % per_tile;
  if (b.col >= p.chunks[0]) {
    b.col -= p.chunks[0];
    b.slice = 1;
    if (b.col >= p.chunks[1]) {
      b.col -= p.chunks[1];
      b.slice = 2;
    }
  }
  b.col *= kLeCols;
  return b;
}

__global__ void __launch_bounds__(kLeThreads, 1)
    expand_long_kernel(const AdapterParams p, const LeCfg cfg, const __grid_constant__ LeMaps maps) {
  extern __shared__ uint8_t s_raw[];
  griddep_wait();
  griddep_launch_dependents();
  uint8_t* smem = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);
  const int h_bytes = 2 * cfg.panels * kLePanel;
  const int stage_bytes = (cfg.panels + 2) * kLePanel;
  uint8_t* ring = smem + cfg.hbufs * h_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kLeBytes);
  uint64_t* empty = full + kLeMaxStages;     // the block's MMAs and the epilogue warps
  uint64_t* h_full = empty + kLeMaxStages;   // [2]
  uint64_t* h_empty = h_full + 2;            // [2]
  uint64_t* acc_full = h_empty + 2;          // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2]
  uint64_t* done = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  int* abort_i = reinterpret_cast<int*>(tmem_holder + 2);
  volatile int* abort_flag = abort_i;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t kTmemCols = 2 * kLeCols;
  if (threadIdx.x == 0) {
    for (int s = 0; s < cfg.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1 + kLeEpilogueWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&h_full[i], 1);
      mbar_init(&h_empty[i], 1);
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kLeEpilogueWarps);
    }
    mbar_init(done, 1);
    *abort_i = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;
  const int64_t total = (int64_t)p.num_segs * (p.chunks[0] + p.chunks[1] + p.chunks[2]);
  const int i0 = (int)(total * blockIdx.x / gridDim.x), i1 = (int)(total * (blockIdx.x + 1) / gridDim.x);
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&maps.h);
      tma_prefetch_desc(&maps.b);
      fence_proxy_async_global();
      int m = -1, tile = -1, slice = -1, adapter = 0, token = 0, b_row = 0, i = i0;   // m: (tile, destination) pairs so far
      for (; i < i1; ++i) {
        const LeBlock blk = le_block(p, i);
        const int g = i - i0, s = g % cfg.stages;
        if (blk.tile != tile || blk.slice != slice) {
          if (blk.tile != tile) {
            const AdapterSeg seg = p.segs[blk.tile];
            adapter = seg.adapter;
            token = seg.token;
          }
          tile = blk.tile;
          slice = blk.slice;
          b_row = adapter * p.N + (slice > 0 ? p.cols[0] : 0) + (slice > 1 ? p.cols[1] : 0);
          const int hb = (m + 1) % cfg.hbufs;
          if (!mbar_wait(&h_empty[hb], (((m + 1) / cfg.hbufs) & 1) ^ 1, abort_flag)) break;
          ++m;
          mbar_arrive_expect_tx(&h_full[hb], (uint32_t)h_bytes);
          for (int term = 0; term < 2; ++term)
            for (int k = 0; k < cfg.panels; ++k)
              tma_load_2d(smem + hb * h_bytes + (term * cfg.panels + k) * kLePanel, &maps.h, &h_full[hb],
                          slice * p.h_slice + k * 64, (term * p.num_segs + tile) * kAdTileRows);
        }
        if (!mbar_wait(&empty[s], ((g / cfg.stages) & 1) ^ 1, abort_flag)) break;
        uint8_t* st = ring + s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], (uint32_t)stage_bytes);
        tma_load_2d(st, &maps.y[slice], &full[s], blk.col, token);
        tma_load_2d(st + kLePanel, &maps.y[slice], &full[s], blk.col + 64, token);
        for (int k = 0; k < cfg.panels; ++k)
          tma_load_2d(st + (2 + k) * kLePanel, &maps.b, &full[s], k * 64, b_row + blk.col);
      }
      // before the CTA exits, what was issued has landed
      const int n = i - i0;
      for (int s = 0; s < cfg.stages && s < n; ++s) drain_wait(&full[s], ((n - 1 - s) / cfg.stages) & 1, abort_flag);
      for (int h = 0; h < cfg.hbufs && h <= m; ++h) drain_wait(&h_full[h], ((m - h) / cfg.hbufs) & 1, abort_flag);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16_f32(kAdTileRows, kLeCols, false);
    int m = -1, tile = -1, slice = -1, rank = 0;
    for (int i = i0; i < i1; ++i) {
      const LeBlock blk = le_block(p, i);
      const int g = i - i0, s = g % cfg.stages, buf = g & 1;
      bool ok = true;
      if (blk.tile != tile || blk.slice != slice) {
        if (blk.tile != tile) rank = rank_of(p, p.segs[blk.tile].adapter);
        tile = blk.tile;
        slice = blk.slice;
        ++m;
        ok = mbar_wait(&h_full[m % cfg.hbufs], (m / cfg.hbufs) & 1, abort_flag);
      }
      ok = ok && mbar_wait(&acc_empty[buf], ((g >> 1) & 1) ^ 1, abort_flag) &&
           mbar_wait(&full[s], (g / cfg.stages) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      uint8_t* rows_b = ring + s * stage_bytes + 2 * kLePanel;
      if (rank % 16) {
        // ranks that the adapter does not have, in the last step: zeros (they may hold anything)
        const int k0 = rank / 8 * 8, kend = (rank + 15) / 16 * 16;
        for (int r = lane; r < kLeCols; r += 32)
          for (int k = k0; k < kend; k += 8) {
            uint16_t* to = reinterpret_cast<uint16_t*>(rows_b + (k / 64) * kLePanel + r * 128 +
                                                       (((k % 64) / 8) ^ (r & 7)) * 16);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (k + e >= rank) to[e] = 0;
          }
        fence_async_shared();
        __syncwarp();
      }
      if (lane == 0) {
        tc_fence_after_sync();
        const uint32_t acc = tmem + (uint32_t)(buf * kLeCols), b = smem_u32(rows_b);
        const uint32_t h = smem_u32(smem + (m % cfg.hbufs) * h_bytes);
        for (int k = 0; k < (rank + 15) / 16; ++k) {
          const uint32_t to = (uint32_t)(k / 4 * kLePanel + k % 4 * 32);
          const uint64_t bd = sdesc_sw128(b + to, 16, 1024);
          tc_mma_bf16(acc, sdesc_sw128(h + to, 16, 1024), bd, idesc, k > 0 ? 1u : 0u);
          tc_mma_bf16(acc, sdesc_sw128(h + (uint32_t)(cfg.panels * kLePanel) + to, 16, 1024), bd, idesc, 1u);
        }
        tc_commit(&empty[s]);
        tc_commit(&acc_full[buf]);
        // (the block after this one belongs to another pair: h may be replaced)
        const LeBlock next = le_block(p, i + 1);
        if (next.tile != tile || next.slice != slice) tc_commit(&h_empty[m % cfg.hbufs]);
      }
      __syncwarp();
    }
    if (lane == 0) {
      // every MMA issued completes before the tensor memory is freed
      tc_commit(done);
      drain_wait(done, 0u, abort_flag);
    }
  } else {
    const int wq = warp & 3, row = wq * 32 + lane, half = warp >= 6 ? 1 : 0;
    int tile = -1, rank = 0, rows = 0;
    int64_t token = 0;
    for (int i = i0; i < i1; ++i) {
      const LeBlock blk = le_block(p, i);
      const int g = i - i0, s = g % cfg.stages, buf = g & 1;
      if (blk.tile != tile) {
        tile = blk.tile;
        const AdapterSeg seg = p.segs[tile];
        rank = rank_of(p, seg.adapter);
        rows = seg.rows;
        token = seg.token;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (g / cfg.stages) & 1, abort_flag) &&
                                       mbar_wait(&acc_full[buf], (g >> 1) & 1, abort_flag)))
        break;
      tc_fence_after_sync();
      uint8_t* panel = ring + s * stage_bytes + half * kLePanel;
      if (rank > 0) {       // (without: y as it is)
        uint32_t v[64];
        const uint32_t acc = tmem + ((uint32_t)(wq * 32) << 16) + (uint32_t)(buf * kLeCols + half * 64);
        tmem_ld32(acc, v);
        tmem_ld32(acc + 32, v + 32);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint4* to = reinterpret_cast<uint4*>(panel + row * 128 + (q ^ (row & 7)) * 16);
          const uint4 y = *to;
          const uint32_t w[4] = {y.x, y.y, y.z, y.w};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = pack_bf16x2(bf16lo_to_f32(w[e]) + __uint_as_float(v[q * 8 + 2 * e]),
                               bf16hi_to_f32(w[e]) + __uint_as_float(v[q * 8 + 2 * e + 1]));
          *to = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
      // the warp's 32 rows, 8 lanes to 128 bytes
      const int cols = p.cols[blk.slice], col = blk.col + half * 64 + (lane & 7) * 8;
      uint16_t* out = p.out[blk.slice] + col;
#pragma unroll
      for (int r8 = 0; r8 < 8; ++r8) {
        const int r = wq * 32 + r8 * 4 + (lane >> 3);
        const uint4 v = *reinterpret_cast<const uint4*>(panel + r * 128 + ((lane & 7) ^ (r & 7)) * 16);
        if (r < rows && col < cols) *reinterpret_cast<uint4*>(out + (token + r) * cols) = v;
      }
      // the sums stood where the next copy lands
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) report_error(p.dev_error, HB_DEVERR_TIMEOUT);
}

}  // namespace hb
