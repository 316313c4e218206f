// adapters.cu -- low-rank adapters of many requests beside a shared projection
// (hb_adapters): each token's row of the projection's output gets its own
// request's product,
//
//   out_i[t] = y_i[t] + scale[a] * (x[t] A_{a,i}^T) B_{a,i}^T,  a = adapter of t,
//
// for up to three destinations i (q, k and v of a fused projection).
//
// With ranks r of 8 to 128 a byte of x, y or an adapter meets about r
// operations where the tensor cores need 284 per byte of HBM: the bytes bound
// it, each row of x and y and each adapter in use moved once from HBM.
//
// The plan (host) sorts the batch's rows by adapter, so that requests of one
// adapter share its reads wherever they stand in the batch, and cuts them into
// long tiles (up to 128 rows that are neighbours in the batch: prompts) and short
// segments (up to 16 rows from anywhere: decodes).  Each kind has its two
// launches, h = x A^T (shrink; fp32 sums, the ranks of all destinations side by
// side) and out = y + scale h B^T (expand; h enters as two bf16 terms, 16 bits of
// it, B's 8 are exact).  The long ones are in adapters_long.cuh.  The short ones
// run on warp MMAs straight from registers, since a decode's 1 to 16 rows fill no
// more of a tensor core tile and every byte of an adapter is used once:
//
//  shrink  A CTA takes a segment and up to 64 ranks; its eight warps (and, where
//          CTAs are too few, several CTAs) cut K among them, so no element is read
//          twice by a CTA and nothing is staged: a lane loads 16 bytes of a row,
//          the order of K inside a product being free as long as both operands
//          have the same.  The warps' sums meet in shared memory, the CTAs' in the
//          next launch.
//  expand  A warp takes 32 columns of B and y at a time, the next 32 on their way;
//          columns are permuted so that a lane's eight results are neighbours and
//          y moves in 16-byte pieces.
//
// Order of the launches of a call with both kinds: shrink long, shrink short,
// expand long, expand short.  The second and the fourth need nothing of the one
// before them: they start under it and wait for it at their end (kWaitLast).
//
// Measured on GB300 (a call among others in a graph, inputs not in L2): 64 decodes,
// 48 adapters of rank 16, K 4096, N 6144 11.6 us (24 MB; 8.4 us from L2: two launches
// of one latency chain each); 64 decodes and a chunk of 448, ranks 8-64, K 14336, N
// 4096 32 us; 5 prompts of 1201 and 61 decodes, ranks 16-64, K 7168, N 9216 100 us.
// All rows in 64-row segments on warp MMAs: 48 and 229 us for the last two.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstring>
#include <mutex>
#include <vector>

#include "adapters.h"
#include "adapters_long.cuh"
#include "hb.h"
#include "hb_internal.h"
#include "operands.h"
#include "ptx.cuh"

namespace hb {

hb_status internal_ok();
hb_status internal_device(int** err, int* num_sms);
hb_status internal_map_2d(CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int box_rows, const char* what);
void internal_count_launch();
void internal_note_other_launch(void* stream);

namespace {

constexpr int kAdThreads = 256, kAdWarps = kAdThreads / 32;
// Neighbouring rows of an adapter from which they are long tiles: a 64-token chunk
// and 4 decodes at K 512 take 4.1 us as short segments, 9.8 us with a tile (four
// launches instead of two).  Measured for that K and rank alone, and not between 64 rows
// and 128.  (A shorter run of more than 16 rows reads its adapter once per segment, from
// L2.)
constexpr int kAdLongRun = 128;
constexpr int kAdGroupRanks = 64;       // ranks that a short shrink CTA holds (at most)
constexpr int kAdShortPieces = 16;      // its pieces of K (at most)
constexpr uint32_t kAdMagic = 0x32414248u;   // "HBA2"

// Host plan = header, then the segments (long tiles, short ones, those of rows
// without an adapter), then the row list (tokens, in the segments' order); the
// latter two are copied to the start of the workspace.
struct AdapterPlan {
  uint32_t magic;
  int32_t num_seqs, total_q, num_adapters, max_ranks, num_sms;
  int32_t num_long, num_short, num_idle;              // segments
  int32_t long_rows, short_rows;                      // rows of the first two
  int32_t short_pieces;                               // pieces of K (at most)
  uint64_t ws_rows, ws_long, ws_short, ws_total, plan_bytes;
};
static_assert(sizeof(AdapterPlan) == 88, "adapter plan header");

__device__ __forceinline__ uint4 ld_nc(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// ---------------------------------------------------------------- shrink
// kN: 8-rank tiles of the CTA.
template <int kN>
__global__ void __launch_bounds__(kAdThreads, 2) shrink_short_kernel(const AdapterParams p) {
  __shared__ float s_sum[kAdWarps * kAdShortRows * kN * 8];
  if (p.wait != kWaitLast) griddep_wait();
  griddep_launch_dependents();
  int at = blockIdx.x;
  const AdapterSeg seg = p.segs[at % p.num_segs];
  at /= p.num_segs;
  const int group = at % p.groups, piece = at / p.groups;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int rank = rank_of(p, seg.adapter);
  float acc[kN][4];
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  // the lane's rows of x and of A (NULL: zeros)
  const uint16_t* xr[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = i * 8 + g;
    xr[i] = r < seg.rows ? p.x + (int64_t)__ldg(p.rows + seg.first + r) * p.K : nullptr;
  }
  const int rank0 = group * p.group_ranks;
  const uint16_t* ar[kN];
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    const int j = rank0 + n * 8 + g;   // of all destinations' ranks
    const bool there = n * 8 + g < p.group_ranks && j < p.ranks && j % p.R < rank;
    ar[n] = there ? p.a + ((int64_t)seg.adapter * p.ranks + j) * p.K : nullptr;
  }
  const int units = (p.K + 63) / 64;
  const int u1 = min(units, (piece + 1) * p.units_per_piece);
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
  for (int u = piece * p.units_per_piece + warp; u < u1; u += kAdWarps) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int k = u * 64 + half * 32 + c * 8;
      const bool in = k < p.K;
      uint4 xv[2], av[kN];
#pragma unroll
      for (int i = 0; i < 2; ++i) xv[i] = in && xr[i] ? ld_nc(xr[i] + k) : zero;
#pragma unroll
      for (int n = 0; n < kN; ++n) av[n] = in && ar[n] ? ld_nc(ar[n] + k) : zero;
      const uint32_t lo[4] = {xv[0].x, xv[1].x, xv[0].y, xv[1].y};
      const uint32_t hi[4] = {xv[0].z, xv[1].z, xv[0].w, xv[1].w};
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        mma_bf16_16816(acc[n], lo, av[n].x, av[n].y);
        mma_bf16_16816(acc[n], hi, av[n].z, av[n].w);
      }
    }
  }
  // the warps' sums, added in their order
  constexpr int kCols = kN * 8;
  float* mine = s_sum + warp * kAdShortRows * kCols;
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float2*>(mine + (i * 8 + g) * kCols + n * 8 + 2 * c) = make_float2(acc[n][2 * i], acc[n][2 * i + 1]);
  __syncthreads();
  for (int t = threadIdx.x; t < kAdShortRows * kCols / 4; t += kAdThreads) {
    const int r = t / (kCols / 4), col = t % (kCols / 4) * 4;
    if (r >= seg.rows || col >= p.group_ranks || rank0 + col >= p.ranks) continue;
    float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < kAdWarps; ++w) {
      const float4 o = *reinterpret_cast<const float4*>(s_sum + (w * kAdShortRows + r) * kCols + col);
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
    *reinterpret_cast<float4*>(p.h + ((int64_t)piece * p.num_rows + seg.first - p.first_row + r) * p.ranks + rank0 + col) = v;
  }
  if (p.wait == kWaitLast) griddep_wait();
}

// ---------------------------------------------------------------- expand
// bf16 pairs of B with the ranks from `rank` on (what an adapter does not have) as zeros
__device__ __forceinline__ uint32_t keep_pair(uint32_t v, int at, int rank) {
  return at + 1 < rank ? v : at < rank ? v & 0xFFFFu : 0u;
}

__global__ void __launch_bounds__(kAdThreads, 2) expand_short_kernel(const AdapterParams p) {
  __shared__ uint4 s_frag[2][kAdMaxRank / 16 * 32];    // [term][step][lane] of h
  if (p.wait == kWaitFirst) griddep_wait();
  if (p.wait != kWaitResults) griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int chunks = p.chunks[0] + p.chunks[1] + p.chunks[2];
  const AdapterSeg seg = p.segs[blockIdx.x / chunks];
  int chunk = blockIdx.x % chunks, slice = 0, first_col = 0;
  while (slice < 2 && chunk >= p.chunks[slice]) {
    chunk -= p.chunks[slice];
    first_col += p.cols[slice];
    ++slice;
  }
  const int cols = p.cols[slice];
  const uint16_t* y = p.y[slice];
  uint16_t* out = p.out[slice];
  const int rank = rank_of(p, seg.adapter);
  // steps of 16 ranks; pairs of steps read 16 bytes of a row of B per lane
  const int steps = (rank + 15) / 16;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  int64_t row[2];   // (-1: no row)
#pragma unroll
  for (int i = 0; i < 2; ++i) row[i] = i * 8 + g < seg.rows ? (int64_t)__ldg(p.rows + seg.first + i * 8 + g) * cols : -1;
  const int end = min(cols, (chunk + 1) * p.chunk_cols);
  int n0 = chunk * p.chunk_cols + warp * 32;
  auto load_y = [&](int n, uint4 (&v)[2]) {
    const int col = n + c * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v[i] = n < end && col < cols && row[i] >= 0 ? *reinterpret_cast<const uint4*>(y + row[i] + col) : zero;
  };
  // the lane's part of B for 32 columns and two steps (or the last one)
  const uint16_t* b = seg.adapter < 0 ? nullptr : p.b + ((int64_t)seg.adapter * p.N + first_col) * p.R;
  auto load_b = [&](int n, int step, uint4 (&v)[4]) {
    const bool two = step + 1 < steps;
    const int base = two ? step * 16 + c * 8 : step * 16 + c * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = n + (g >> 1) * 8 + 2 * j + (g & 1);
      v[j] = zero;
      if (n < end && col < cols && base < rank) {
        const uint16_t* src = b + (int64_t)col * p.R + base;
        if (two) v[j] = ld_nc(src);
        else {
          const uint2 o = __ldg(reinterpret_cast<const uint2*>(src));
          v[j].x = o.x;
          v[j].y = o.y;
        }
      }
    }
  };
  uint4 yn[2], bn[4];      // what comes next
  load_y(n0, yn);
  if (rank > 0) load_b(n0, 0, bn);
  if (p.wait == kWaitResults) {
    griddep_wait();
    griddep_launch_dependents();
  }
  if (rank > 0) {
    const float scale = __ldg(p.scale + seg.adapter);
    for (int t = threadIdx.x; t < steps * 32; t += kAdThreads) {
      const int l = t & 31, step = t >> 5;
      const bool paired = step < (steps & ~1);
      const int base = paired ? (step >> 1) * 32 + (l & 3) * 8 + (step & 1) * 4 : step * 16 + (l & 3) * 4;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = i * 8 + (l >> 2);
        float4 v = make_float4(0, 0, 0, 0);
        if (r < seg.rows && base < p.R) {
          const float* src = p.h + (int64_t)(seg.first - p.first_row + r) * p.ranks + slice * p.R + base;
#pragma unroll 8
          for (int piece = 0; piece < p.pieces; ++piece) {
            const float4 o = __ldcg(reinterpret_cast<const float4*>(src + (int64_t)piece * p.num_rows * p.ranks));
            v.x += o.x;
            v.y += o.y;
            v.z += o.z;
            v.w += o.w;
          }
        }
        // (a rank that the adapter does not have may have met an infinity of x)
        two_terms(base < rank ? v.x * scale : 0.f, base + 1 < rank ? v.y * scale : 0.f, hi[i], lo[i]);
        two_terms(base + 2 < rank ? v.z * scale : 0.f, base + 3 < rank ? v.w * scale : 0.f, hi[i + 2], lo[i + 2]);
      }
      s_frag[0][t] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      s_frag[1][t] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  __syncthreads();
  constexpr int kStride = kAdWarps * 32;
  for (; n0 < end; n0 += kStride) {
    uint4 yv[2] = {yn[0], yn[1]};
    float acc[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    load_y(n0 + kStride, yn);
    for (int step = 0; step < steps; step += 2) {
      const bool two = step + 1 < steps;
      const int base = two ? step * 16 + c * 8 : step * 16 + c * 4;
      uint4 bv[4] = {bn[0], bn[1], bn[2], bn[3]};
      if (step + 2 < steps) load_b(n0, step + 2, bn);
      else load_b(n0 + kStride, 0, bn);
      if (base + (two ? 8 : 4) > rank) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bv[j].x = keep_pair(bv[j].x, base, rank);
          bv[j].y = keep_pair(bv[j].y, base + 2, rank);
          bv[j].z = keep_pair(bv[j].z, base + 4, rank);
          bv[j].w = keep_pair(bv[j].w, base + 6, rank);
        }
      }
#pragma unroll
      for (int term = 0; term < 2; ++term) {
        const uint4 v = s_frag[term][step * 32 + lane];
        const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_bf16_16816(acc[j], a, bv[j].x, bv[j].y);
      }
      if (!two) continue;
#pragma unroll
      for (int term = 0; term < 2; ++term) {
        const uint4 v = s_frag[term][(step + 1) * 32 + lane];
        const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_bf16_16816(acc[j], a, bv[j].z, bv[j].w);
      }
    }
    const int col = n0 + c * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (col >= cols || row[i] < 0) continue;
      uint32_t v[4] = {yv[i].x, yv[i].y, yv[i].z, yv[i].w};
      if (rank > 0) {       // (without: the bytes as they are)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = pack_bf16x2(bf16lo_to_f32(v[j]) + acc[j][2 * i], bf16hi_to_f32(v[j]) + acc[j][2 * i + 1]);
      }
      *reinterpret_cast<uint4*>(out + row[i] + col) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  if (p.wait == kWaitLast) griddep_wait();
}

// ---------------------------------------------------------------- launches
cudaError_t launch_shrink_short(const AdapterParams& p, cudaStream_t st) {
  const unsigned grid = (unsigned)p.num_segs * p.groups * p.pieces;
  const int n = (p.group_ranks + 7) / 8;
  auto kernel = n <= 1   ? shrink_short_kernel<1>
                : n <= 2 ? shrink_short_kernel<2>
                : n <= 4 ? shrink_short_kernel<4>
                : n <= 6 ? shrink_short_kernel<6>
                         : shrink_short_kernel<8>;
  return launch_serialized(kernel, grid, kAdThreads, 0, st, p);
}

// Chunks of columns, in whole rounds of the CTA's warps: few rounds of CTAs over
// the SMs (two at a time each) of few rounds of columns.
cudaError_t launch_expand_short(AdapterParams p, int num_sms, cudaStream_t st) {
  constexpr int kRound = kAdWarps * 32;
  const int most = (*std::max_element(p.cols, p.cols + 3) + kRound - 1) / kRound;
  int best = 1;
  double best_cost = 0;
  for (int rounds = 1; rounds <= std::min(most, 64); ++rounds) {
    int64_t chunks = 0;
    for (int i = 0; i < 3; ++i) chunks += (p.cols[i] + rounds * kRound - 1) / (rounds * kRound);
    const double cost = (double)((p.num_segs * chunks + 2 * num_sms - 1) / (2 * num_sms)) * (rounds + 3);
    if (rounds == 1 || cost < best_cost) best = rounds, best_cost = cost;
  }
  p.chunk_cols = best * kRound;
  int64_t chunks = 0;
  for (int i = 0; i < 3; ++i) chunks += p.chunks[i] = (p.cols[i] + p.chunk_cols - 1) / p.chunk_cols;
  if (p.num_segs * chunks > INT_MAX) return cudaErrorInvalidConfiguration;
  return launch_serialized(expand_short_kernel, (unsigned)(p.num_segs * chunks), kAdThreads, 0, st, p);
}

cudaLaunchConfig_t shrink_long_config(int ctas, int pieces, cudaStream_t st, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kLsThreads);
  cfg.dynamicSmemBytes = kLsSmem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)pieces;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters of 1 .. kLsMaxPieces CTAs that the device holds at a time (a cluster's
// CTAs sit in one group of SMs, so these are fewer than SMs / CTAs); found once
// per device.
struct Clusters {
  int fit[kLsMaxPieces + 1];
};
cudaError_t clusters_of_device(const Clusters** out) {
  static std::mutex mu;
  static Clusters per_device[64];
  static bool ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(shrink_long_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLsSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(shrink_long_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    for (int n = 1; e == cudaSuccess && n <= kLsMaxPieces; ++n) {
      cudaLaunchAttribute attr[2];
      cudaLaunchConfig_t cfg = shrink_long_config(n, n, nullptr, attr);
      cfg.attrs = attr + 1;   // (the cluster's size alone)
      cfg.numAttrs = 1;
      int fit = 0;
      e = cudaOccupancyMaxActiveClusters(&fit, shrink_long_kernel, &cfg);
      per_device[dev].fit[n] = fit;
    }
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  *out = &per_device[dev];
  return cudaSuccess;
}

cudaError_t launch_shrink_long(const AdapterParams& p, const CUtensorMap& xmap, const CUtensorMap& amap, cudaStream_t st) {
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = shrink_long_config(p.num_segs * p.groups * p.pieces, p.pieces, st, attr);
  return cudaLaunchKernelEx(&cfg, shrink_long_kernel, p, xmap, amap);
}

cudaError_t launch_expand_long(const AdapterParams& p, const LeMaps& maps, int num_sms, cudaStream_t st) {
  const cudaError_t e =
      cudaFuncSetAttribute(expand_long_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLeSmem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (int64_t)p.num_segs * (p.chunks[0] + p.chunks[1] + p.chunks[2]);
  return launch_serialized(expand_long_kernel, (unsigned)std::min<int64_t>(blocks, num_sms), kLeThreads, kLeSmem, st, p,
                           le_cfg(p.R), maps);
}

}  // namespace
}  // namespace hb

using namespace hb;

extern "C" hb_status hb_adapters_plan(int32_t num_seqs, int32_t total_q, const int32_t* h_q_len,
                                      const int32_t* h_adapter, int32_t num_adapters, int32_t max_ranks,
                                      int32_t num_sms, void* h_plan, size_t* plan_bytes, void* d_workspace,
                                      size_t* workspace_bytes, void* stream) {
  try {
    if (!plan_bytes || !workspace_bytes)
      return internal_fail(HB_ERR_INVALID_ARG, "plan_bytes and workspace_bytes must be non-NULL");
    if (num_seqs < 0 || total_q < 0 || num_adapters <= 0 || num_sms <= 0)
      return internal_failf(HB_ERR_SHAPE, "num_seqs %d, total_q %d, num_adapters %d, num_sms %d", num_seqs, total_q,
                            num_adapters, num_sms);
    if (max_ranks <= 0 || max_ranks > 3 * kAdMaxRank || max_ranks % 8)
      return internal_failf(HB_ERR_SHAPE, "max_ranks %d: a multiple of 8 up to %d", max_ranks, 3 * kAdMaxRank);
    if (num_seqs > 0 && (!h_q_len || !h_adapter))
      return internal_fail(HB_ERR_INVALID_ARG, "h_q_len and h_adapter must be non-NULL");
    // the runs of neighbouring rows of one adapter; what each adapter has outside of long ones
    struct Run {
      int32_t adapter, token, rows;
    };
    thread_local std::vector<Run> runs;
    thread_local std::vector<int32_t> count, list;
    thread_local std::vector<AdapterSeg> segs;
    runs.clear();
    int64_t tokens = 0;
    for (int32_t s = 0; s < num_seqs; ++s) {
      if (h_q_len[s] < 0) return internal_failf(HB_ERR_SHAPE, "sequence %d: q_len %d", s, h_q_len[s]);
      if (h_adapter[s] < -1 || h_adapter[s] >= num_adapters)
        return internal_failf(HB_ERR_SHAPE, "sequence %d: adapter %d of %d", s, h_adapter[s], num_adapters);
      if (tokens + h_q_len[s] > total_q)
        return internal_failf(HB_ERR_SHAPE, "the sequences have more than total_q (%d) tokens", total_q);
      if (h_q_len[s] == 0) continue;
      if (!runs.empty() && runs.back().adapter == h_adapter[s]) runs.back().rows += h_q_len[s];
      else runs.push_back({h_adapter[s], (int32_t)tokens, h_q_len[s]});
      tokens += h_q_len[s];
    }
    AdapterPlan h{};
    segs.clear();
    list.resize((size_t)tokens);
    count.assign((size_t)num_adapters + 1, 0);     // [a + 1]: rows of a in short runs ([0]: without)
    int32_t at = 0;
    for (const Run& r : runs) {
      if (r.adapter < 0 || r.rows < kAdLongRun) {
        count[r.adapter + 1] += r.rows;
        continue;
      }
      // tiles of like length
      const int32_t tiles = (r.rows + kAdTileRows - 1) / kAdTileRows;
      const int32_t per = ((r.rows + tiles - 1) / tiles + 15) / 16 * 16;
      for (int32_t i = 0; i < r.rows; i += per)
        segs.push_back({r.adapter, at + i, std::min(per, r.rows - i), r.token + i});
      for (int32_t i = 0; i < r.rows; ++i) list[at++] = r.token + i;
    }
    h.num_long = (int32_t)segs.size();
    h.long_rows = at;
    // the others by adapter (counting sort), those without one last
    auto cut = [&](int32_t a) {
      const int32_t n = count[a + 1];
      for (int32_t i = 0; i < n; i += kAdShortRows) segs.push_back({a, at + i, std::min(kAdShortRows, n - i), -1});
      count[a + 1] = at;
      at += n;
    };
    for (int32_t a = 0; a < num_adapters; ++a) cut(a);
    h.num_short = (int32_t)segs.size() - h.num_long;
    h.short_rows = at - h.long_rows;
    cut(-1);
    h.num_idle = (int32_t)segs.size() - h.num_long - h.num_short;
    for (const Run& r : runs)
      if (r.adapter < 0 || r.rows < kAdLongRun)
        for (int32_t i = 0; i < r.rows; ++i) list[count[r.adapter + 1]++] = r.token + i;
    auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
    h.magic = kAdMagic;
    h.num_seqs = num_seqs;
    h.total_q = total_q;
    h.num_adapters = num_adapters;
    h.max_ranks = max_ranks;
    h.num_sms = num_sms;
    // pieces of K that fill the SMs twice
    h.short_pieces =
        h.num_short ? std::min(kAdShortPieces, std::max(1, (2 * num_sms + h.num_short - 1) / h.num_short)) : 1;
    h.ws_rows = segs.size() * sizeof(AdapterSeg);
    const uint64_t items = h.ws_rows + (uint64_t)tokens * 4;
    h.ws_long = up(items);
    // (each destination's ranks in whole steps of 16: 8 more at most)
    h.ws_short = up(h.ws_long + 4ull * h.num_long * kAdTileRows * (max_ranks + 24));
    h.ws_total = up(h.ws_short + (uint64_t)h.short_pieces * h.short_rows * max_ranks * 4);
    h.plan_bytes = sizeof(h) + items;
    const size_t have_plan = *plan_bytes, have_ws = *workspace_bytes;
    *plan_bytes = h.plan_bytes;
    *workspace_bytes = h.ws_total;
    if (!h_plan) return internal_ok();
    if (have_plan < h.plan_bytes)
      return internal_failf(HB_ERR_WORKSPACE, "plan buffer has %zu bytes, needs %zu", have_plan, (size_t)h.plan_bytes);
    if (d_workspace) {
      if (have_ws < h.ws_total)
        return internal_failf(HB_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have_ws, (size_t)h.ws_total);
      if (reinterpret_cast<uintptr_t>(d_workspace) & 255u)
        return internal_fail(HB_ERR_INVALID_ARG, "d_workspace must be 256-byte aligned");
    }
    uint8_t* to = static_cast<uint8_t*>(h_plan);
    std::memcpy(to, &h, sizeof(h));
    uint8_t* body = to + sizeof(h);
    if (!segs.empty()) std::memcpy(body, segs.data(), h.ws_rows);
    if (!list.empty()) std::memcpy(body + h.ws_rows, list.data(), list.size() * 4);
    if (!d_workspace || items == 0) return internal_ok();
    const cudaError_t e =
        cudaMemcpyAsync(d_workspace, body, items, cudaMemcpyHostToDevice, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return internal_failf(HB_ERR_CUDA, "plan upload: %s", cudaGetErrorString(e));
    return internal_ok();
  } catch (...) {
    return internal_fail(HB_ERR_CUDA, "unexpected exception in hb_adapters_plan");
  }
}

extern "C" hb_status hb_adapters(const hb_adapter_pool* pool, const void* h_plan, const void* x,
                                 const hb_linear_out* y, const hb_linear_out* out, void* d_workspace, void* stream) {
  try {
    if (!pool || !h_plan || !y || !out)
      return internal_fail(HB_ERR_INVALID_ARG, "pool, h_plan, y and out must be non-NULL");
    AdapterPlan h;
    std::memcpy(&h, h_plan, sizeof(h));
    if (h.magic != kAdMagic) return internal_fail(HB_ERR_WORKSPACE, "h_plan is not a plan written by hb_adapters_plan");
    const int R = pool->max_rank, K = pool->K, N = pool->N, slices = pool->slices;
    if (pool->num_adapters <= 0 || K <= 0 || N <= 0 || slices < 1 || slices > 3)
      return internal_failf(HB_ERR_SHAPE, "pool: num_adapters %d, K %d, N %d, slices %d", pool->num_adapters, K, N, slices);
    if (R <= 0 || R % 8 || R > kAdMaxRank)
      return internal_failf(HB_ERR_UNSUPPORTED, "max_rank %d: a multiple of 8 up to %d", R, kAdMaxRank);
    if (K % 8) return internal_failf(HB_ERR_UNSUPPORTED, "K %d: a multiple of 8 is needed", K);
    if ((int64_t)pool->num_adapters * std::max((int64_t)N, (int64_t)slices * R) > INT_MAX)
      return internal_failf(HB_ERR_UNSUPPORTED, "%d adapters are too many", pool->num_adapters);
    if (h.num_adapters != pool->num_adapters || h.max_ranks < slices * R)
      return internal_failf(HB_ERR_WORKSPACE, "plan of %d adapters and %d ranks, the pool has %d and %d", h.num_adapters,
                            h.max_ranks, pool->num_adapters, slices * R);
    int64_t sum = 0;
    for (int i = 0; i < 3; ++i) {
      if (y->cols[i] != out->cols[i] || y->cols[i] < 0 || (y->cols[i] > 0) != (i < slices))
        return internal_failf(HB_ERR_SHAPE, "cols[%d]: y has %d, out %d, the pool %d destinations", i, y->cols[i],
                              out->cols[i], slices);
      if (y->cols[i] % 8) return internal_failf(HB_ERR_UNSUPPORTED, "cols[%d] = %d: multiples of 8 needed", i, y->cols[i]);
      sum += y->cols[i];
    }
    if (sum != N) return internal_failf(HB_ERR_SHAPE, "cols sum to %lld, N is %d", (long long)sum, N);
    if (h.total_q == 0) return internal_ok();
    if (!pool->rank || !pool->scale) return internal_fail(HB_ERR_INVALID_ARG, "rank and scale must be non-NULL");
    if ((reinterpret_cast<uintptr_t>(pool->rank) | reinterpret_cast<uintptr_t>(pool->scale)) & 3u)
      return internal_fail(HB_ERR_INVALID_ARG, "rank and scale must be 4-byte aligned");
    if (!d_workspace || (reinterpret_cast<uintptr_t>(d_workspace) & 255u))
      return internal_fail(HB_ERR_INVALID_ARG, "d_workspace must be non-NULL and 256-byte aligned");
    const int64_t T = h.total_q, n = pool->num_adapters;
    static const char* const names[2][3] = {{"y[0]", "y[1]", "y[2]"}, {"out[0]", "out[1]", "out[2]"}};
    Operand in[9] = {{x, T, 2LL * K, 2LL * K, "x"},
                     {pool->a, 1, 2 * n * slices * R * K, 0, "a"},
                     {pool->b, 1, 2 * n * N * R, 0, "b"},
                     {pool->rank, 1, 4 * n, 0, "rank"},
                     {pool->scale, 1, 4 * n, 0, "scale"},
                     {d_workspace, 1, (int64_t)h.ws_total, 0, "the workspace"}};
    hb_status s;
    for (int i = 0; i < 3; ++i)
      if ((s = check_rows(in[i])) != HB_OK) return s;
    int num_in = 6;
    bool in_place = true;
    for (int i = 0; i < slices; ++i) {
      in[num_in] = {y->y[i], T, 2LL * y->cols[i], 2LL * y->cols[i], names[0][i]};
      if ((s = check_rows(in[num_in++])) != HB_OK) return s;
      in_place = in_place && y->y[i] == out->y[i];
    }
    for (int i = 0; i < slices; ++i) {
      const Operand o{out->y[i], T, 2LL * out->cols[i], 2LL * out->cols[i], names[1][i]};
      if ((s = check_rows(o)) != HB_OK) return s;
      for (int j = 0; j < num_in; ++j)
        if ((s = check_apart(o, in[j], j == 6 + i)) != HB_OK) return s;
      for (int j = 0; j < i; ++j)
        if ((s = check_apart(o, {out->y[j], T, 2LL * out->cols[j], 2LL * out->cols[j], names[1][j]}, false)) != HB_OK)
          return s;
    }
    // (the workspace is written, with x A^T)
    for (int j = 0; j < num_in; ++j)
      if (j != 5 && (s = check_apart(in[5], in[j], false)) != HB_OK) return s;
    AdapterParams p{};
    int num_sms = 0;
    if ((s = internal_device(&p.dev_error, &num_sms)) != HB_OK) return s;
    uint8_t* ws = static_cast<uint8_t*>(d_workspace);
    const AdapterSeg* segs = reinterpret_cast<const AdapterSeg*>(ws);
    p.rows = reinterpret_cast<const int32_t*>(ws + h.ws_rows);
    p.K = K;
    p.R = R;
    p.slices = slices;
    p.N = N;
    p.ranks = slices * R;
    p.x = static_cast<const uint16_t*>(x);
    p.a = static_cast<const uint16_t*>(pool->a);
    p.b = static_cast<const uint16_t*>(pool->b);
    p.rank = pool->rank;
    p.scale = pool->scale;
    for (int i = 0; i < 3; ++i) {
      p.y[i] = static_cast<const uint16_t*>(y->y[i]);
      p.out[i] = static_cast<uint16_t*>(out->y[i]);
      p.cols[i] = y->cols[i];
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int units = (K + 63) / 64;
    auto cut_k = [&](AdapterParams& q, int pieces) {
      q.units_per_piece = (units + pieces - 1) / pieces;
      q.pieces = (units + q.units_per_piece - 1) / q.units_per_piece;
    };
    auto launched = [&](cudaError_t e) {
      if (e != cudaSuccess) return internal_failf(HB_ERR_CUDA, "adapter launch: %s", cudaGetErrorString(e));
      internal_note_other_launch(stream);
      internal_count_launch();
      return HB_OK;
    };
    AdapterParams lo = p, sh = p;
    lo.segs = segs;
    lo.num_segs = h.num_long;
    lo.num_rows = h.long_rows;
    lo.terms = reinterpret_cast<uint16_t*>(ws + h.ws_long);
    lo.h_slice = (R + 15) / 16 * 16;
    lo.h_cols = slices * lo.h_slice;
    sh.segs = segs + h.num_long;
    sh.num_segs = h.num_short;
    sh.num_rows = h.short_rows;
    sh.first_row = h.long_rows;
    sh.h = reinterpret_cast<float*>(ws + h.ws_short);
    if (h.num_long > 0) {
      // 16-rank boxes per CTA; K cut so that the CTAs' rounds over the SMs are short
      const int boxes = slices * ((R + 15) / 16);
      lo.groups = (boxes + kLsMaxBoxes - 1) / kLsMaxBoxes;
      lo.boxes = (boxes + lo.groups - 1) / lo.groups;
      const int64_t ctas = (int64_t)h.num_long * lo.groups;
      const Clusters* clusters = nullptr;
      const cudaError_t e = clusters_of_device(&clusters);
      if (e != cudaSuccess) return internal_failf(HB_ERR_CUDA, "adapter clusters: %s", cudaGetErrorString(e));
      int best = 1;
      int64_t best_cost = INT64_MAX;
      // (a CTA's start, the sums' exchange and its end take as long as 16 units)
      for (int n = 1; n <= std::min(kLsMaxPieces, units); ++n) {
        if (clusters->fit[n] == 0) continue;
        const int64_t waves = (ctas + clusters->fit[n] - 1) / clusters->fit[n];
        const int64_t cost = waves * ((units + n - 1) / n + 16);
        if (cost < best_cost) best = n, best_cost = cost;
      }
      cut_k(lo, best);
      int64_t blocks = 0;
      for (int i = 0; i < 3; ++i) blocks += lo.chunks[i] = (lo.cols[i] + kLeCols - 1) / kLeCols;
      if (ctas * lo.pieces > INT_MAX || h.num_long * blocks > INT_MAX)
        return internal_fail(HB_ERR_UNSUPPORTED, "too many tokens at once");
    }
    if (h.num_short > 0) {
      sh.groups = (p.ranks + kAdGroupRanks - 1) / kAdGroupRanks;
      sh.group_ranks = ((p.ranks + sh.groups - 1) / sh.groups + 7) / 8 * 8;
      const int64_t ctas = (int64_t)h.num_short * sh.groups;
      // (rounds of two CTAs per SM, one beside a long tile's, each as long as its warps' units and three more)
      const int64_t long_ctas = h.num_long ? (int64_t)h.num_long * lo.groups * lo.pieces : 0;
      const int64_t slots = 2LL * h.num_sms - std::min<int64_t>(h.num_sms, long_ctas);
      int best = 1;
      int64_t best_cost = INT64_MAX;
      for (int n = 1; n <= std::min(h.short_pieces, std::max(1, units / kAdWarps)); ++n) {
        const int64_t rounds = (ctas * n + slots - 1) / slots;
        const int64_t cost = rounds * (((units + n - 1) / n + kAdWarps - 1) / kAdWarps + 3);
        if (cost < best_cost) best = n, best_cost = cost;
      }
      cut_k(sh, best);
      if (ctas * sh.pieces > INT_MAX) return internal_fail(HB_ERR_UNSUPPORTED, "too many tokens at once");
    }
    LeMaps maps{};
    CUtensorMap xmap, amap;
    if (h.num_long > 0) {
      if ((s = internal_map_2d(&xmap, x, K, T, kAdTileRows, "adapter x")) != HB_OK) return s;
      if ((s = internal_map_2d(&amap, pool->a, K, n * slices * R, 16, "adapter a")) != HB_OK) return s;
      if ((s = internal_map_2d(&maps.h, lo.terms, lo.h_cols, 2LL * h.num_long * kAdTileRows, kAdTileRows, "adapter h")) != HB_OK)
        return s;
      if ((s = internal_map_2d(&maps.b, pool->b, R, n * N, kLeCols, "adapter b")) != HB_OK) return s;
      for (int i = 0; i < slices; ++i)
        if ((s = internal_map_2d(&maps.y[i], lo.y[i], lo.cols[i], T, kAdTileRows, "adapter y")) != HB_OK) return s;
    }
    // shrink
    if (h.num_long > 0 && (s = launched(launch_shrink_long(lo, xmap, amap, st))) != HB_OK) return s;
    sh.wait = h.num_long > 0 ? kWaitLast : kWaitFirst;
    if (h.num_short > 0 && (s = launched(launch_shrink_short(sh, st))) != HB_OK) return s;
    // expand; in place, rows without an adapter have nothing to do
    if (h.num_long > 0 && (s = launched(launch_expand_long(lo, maps, h.num_sms, st))) != HB_OK) return s;
    sh.wait = h.num_long > 0 ? kWaitLast : h.num_short > 0 ? kWaitResults : kWaitFirst;
    if (!in_place) sh.num_segs += h.num_idle;
    if (sh.num_segs > 0 && (s = launched(launch_expand_short(sh, h.num_sms, st))) != HB_OK) return s;
    return internal_ok();
  } catch (...) {
    return internal_fail(HB_ERR_CUDA, "unexpected exception in hb_adapters");
  }
}
