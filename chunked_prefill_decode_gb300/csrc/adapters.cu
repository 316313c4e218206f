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
// it, each row of x and y and each adapter in use moved once, and both products
// run on warp MMAs straight from registers.  Two launches:
//
//  shrink  h = x A^T (fp32, ranks of all destinations side by side).  A CTA takes
//          up to 64 rows of one adapter and up to 64 ranks; its eight warps
//          (and, where CTAs are too few, several CTAs) cut K among them, so no
//          element of x or A is read twice by a CTA and nothing is staged: a
//          lane loads 16 bytes of a row, the order of K inside a product being
//          free as long as both operands have the same.  The warps' sums meet
//          in shared memory, the CTAs' in the next launch.
//  expand  out = y + scale h B^T.  h is split into two bf16 terms (16 bits of it
//          enter the product, B's 8 are exact) in the layout of the MMA's
//          operand; a warp takes 32 columns of B and y at a time, columns
//          permuted so that a lane's eight results are neighbours and y moves
//          in 16-byte pieces.
//
// The plan (host) sorts the batch's rows by adapter and cuts them into segments
// of one adapter: requests of one adapter share its reads wherever they stand in
// the batch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <vector>

#include "hb.h"
#include "hb_internal.h"
#include "operands.h"
#include "ptx.cuh"

namespace hb {

hb_status internal_ok();
hb_status internal_device(int** err, int* num_sms);
void internal_count_launch();
void internal_note_other_launch(void* stream);

namespace {

constexpr int kAdThreads = 256, kAdWarps = kAdThreads / 32;
constexpr int kAdSegRows = 64;          // rows of a segment (at most)
constexpr int kAdGroupRanks = 64;       // ranks that a shrink CTA holds (at most)
constexpr int kAdMaxPieces = 16;        // pieces of K (at most)
constexpr int kAdMaxRank = 128;
constexpr uint32_t kAdMagic = 0x31414248u;   // "HBA1"

struct AdapterSeg {
  int32_t adapter;      // -1: rows without one
  int32_t first;        // of the row list
  int32_t rows;
  int32_t pad;
};

// Host plan = header, then the segments (with an adapter first, longest first),
// then the row list (tokens, in the segments' order); the latter two are copied
// to the start of the workspace.
struct AdapterPlan {
  uint32_t magic;
  int32_t num_seqs, total_q, num_adapters, max_ranks, num_sms;
  int32_t num_segs, num_idle_segs;    // with, without an adapter
  int32_t num_rows, max_seg_rows;     // with an adapter
  int32_t max_pieces, pad;
  uint64_t ws_rows, ws_h, ws_total, plan_bytes;
};
static_assert(sizeof(AdapterPlan) == 80, "adapter plan header");

struct AdapterParams {
  const AdapterSeg* segs;
  const int32_t* rows;
  int32_t num_segs, num_rows;
  int32_t K, R, slices, N, ranks;      // ranks = slices * R
  const uint16_t *x, *a, *b;
  const int32_t* rank;
  const float* scale;
  float* h;                            // [pieces, num_rows, ranks]
  int32_t pieces, units_per_piece;     // units: 64 elements of K
  int32_t groups, group_ranks;
  const uint16_t* y[3];
  uint16_t* out[3];
  int32_t cols[3];
  int32_t chunks[3], chunk_cols;       // column chunks per destination
};

__device__ __forceinline__ uint4 ld_nc(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// ranks read as if held to [0, R]
__device__ __forceinline__ int rank_of(const AdapterParams& p, int adapter) {
  return adapter < 0 ? 0 : min(max(__ldg(p.rank + adapter), 0), p.R);
}

// ---------------------------------------------------------------- shrink
// kM: 16-row tiles, kN: 8-rank tiles of the CTA.
template <int kM, int kN>
__device__ void shrink_body(const AdapterParams& p, const AdapterSeg& seg, int group, int piece, float* s_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int rank = rank_of(p, seg.adapter);
  float acc[kM][kN][4];
#pragma unroll
  for (int m = 0; m < kM; ++m)
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][n][e] = 0.f;
  // the lane's rows of x and of A (NULL: zeros)
  const uint16_t* xr[kM][2];
#pragma unroll
  for (int m = 0; m < kM; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = m * 16 + i * 8 + g;
      xr[m][i] = r < seg.rows ? p.x + (int64_t)__ldg(p.rows + seg.first + r) * p.K : nullptr;
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
      uint4 xv[kM][2], av[kN];
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) xv[m][i] = in && xr[m][i] ? ld_nc(xr[m][i] + k) : zero;
#pragma unroll
      for (int n = 0; n < kN; ++n) av[n] = in && ar[n] ? ld_nc(ar[n] + k) : zero;
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const uint32_t lo[4] = {xv[m][0].x, xv[m][1].x, xv[m][0].y, xv[m][1].y};
        const uint32_t hi[4] = {xv[m][0].z, xv[m][1].z, xv[m][0].w, xv[m][1].w};
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          mma_bf16_16816(acc[m][n], lo, av[n].x, av[n].y);
          mma_bf16_16816(acc[m][n], hi, av[n].z, av[n].w);
        }
      }
    }
  }
  // the warps' sums, added in their order
  constexpr int kRows = kM * 16, kCols = kN * 8;
  float* mine = s_sum + warp * kRows * kCols;
#pragma unroll
  for (int m = 0; m < kM; ++m)
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<float2*>(mine + (m * 16 + i * 8 + g) * kCols + n * 8 + 2 * c) =
            make_float2(acc[m][n][2 * i], acc[m][n][2 * i + 1]);
  __syncthreads();
  for (int t = threadIdx.x; t < kRows * kCols / 4; t += kAdThreads) {
    const int r = t / (kCols / 4), col = t % (kCols / 4) * 4;
    if (r >= seg.rows || col >= p.group_ranks || rank0 + col >= p.ranks) continue;
    float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < kAdWarps; ++w) {
      const float4 o = *reinterpret_cast<const float4*>(s_sum + (w * kRows + r) * kCols + col);
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
    *reinterpret_cast<float4*>(p.h + ((int64_t)piece * p.num_rows + seg.first + r) * p.ranks + rank0 + col) = v;
  }
}

template <int kM, int kN>
__global__ void __launch_bounds__(kAdThreads) shrink_kernel(const AdapterParams p) {
  extern __shared__ float4 s_dyn[];
  griddep_wait();
  griddep_launch_dependents();
  int at = blockIdx.x;
  const AdapterSeg seg = p.segs[at % p.num_segs];
  at /= p.num_segs;
  const int group = at % p.groups, piece = at / p.groups;
  float* s_sum = reinterpret_cast<float*>(s_dyn);
  if (kM > 1 && seg.rows <= 16) shrink_body<1, kN>(p, seg, group, piece, s_sum);
  else shrink_body<kM, kN>(p, seg, group, piece, s_sum);
}

// ---------------------------------------------------------------- expand
// bf16 pairs of B with the ranks from `rank` on (what an adapter does not have) as zeros
__device__ __forceinline__ uint32_t keep_pair(uint32_t v, int at, int rank) {
  return at + 1 < rank ? v : at < rank ? v & 0xFFFFu : 0u;
}

// a and b as bf16 pairs hi + lo (what is not finite is hi alone)
__device__ __forceinline__ void two_terms(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  const float ra = a - bf16lo_to_f32(hi), rb = b - bf16hi_to_f32(hi);
  lo = pack_bf16x2(isfinite(ra) ? ra : 0.f, isfinite(rb) ? rb : 0.f);
}

// kM: 16-row tiles at a time
template <int kM>
__global__ void __launch_bounds__(kAdThreads, 2) expand_kernel(const AdapterParams p) {
  extern __shared__ uint4 s_frag[];    // [tile][step][lane] of h: first terms, then second terms
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  int chunks = p.chunks[0] + p.chunks[1] + p.chunks[2];
  const AdapterSeg seg = p.segs[blockIdx.x / chunks];
  int chunk = blockIdx.x % chunks, slice = 0, first_col = 0;
  while (chunk >= p.chunks[slice]) {
    chunk -= p.chunks[slice];
    first_col += p.cols[slice];
    ++slice;
  }
  const int cols = p.cols[slice];
  const uint16_t* y = p.y[slice];
  uint16_t* out = p.out[slice];
  const int rank = rank_of(p, seg.adapter);
  // steps of 16 ranks; pairs of steps read 16 bytes of a row of B per lane
  const int steps = (rank + 15) / 16, tiles = (seg.rows + 15) / 16;
  const int frags = tiles * steps * 32;
  if (rank > 0) {
    const float scale = __ldg(p.scale + seg.adapter);
    for (int t = threadIdx.x; t < frags; t += kAdThreads) {
      const int l = t & 31, step = (t >> 5) % steps, tile = (t >> 5) / steps;
      const bool paired = step < (steps & ~1);
      const int base = paired ? (step >> 1) * 32 + (l & 3) * 8 + (step & 1) * 4 : step * 16 + (l & 3) * 4;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = tile * 16 + i * 8 + (l >> 2);
        float4 v = make_float4(0, 0, 0, 0);
        if (r < seg.rows && base < p.R) {
          const float* src = p.h + (int64_t)(seg.first + r) * p.ranks + slice * p.R + base;
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
      s_frag[t] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      s_frag[frags + t] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  __syncthreads();
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint16_t* b = seg.adapter < 0 ? nullptr : p.b + ((int64_t)seg.adapter * p.N + first_col) * p.R;
  for (int tile0 = 0; tile0 < tiles; tile0 += kM) {
    int64_t row[kM][2];   // (-1: no row)
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (tile0 + m) * 16 + i * 8 + g;
        row[m][i] = r < seg.rows ? (int64_t)__ldg(p.rows + seg.first + r) * cols : -1;
      }
    const int end = min(cols, (chunk + 1) * p.chunk_cols);
    for (int n0 = chunk * p.chunk_cols + warp * 32; n0 < end; n0 += kAdWarps * 32) {
      const int col = n0 + c * 8;
      const bool in = col < cols;
      uint4 yv[kM][2];
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          yv[m][i] = in && row[m][i] >= 0 ? *reinterpret_cast<const uint4*>(y + row[m][i] + col) : zero;
      float acc[kM][4][4];
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
      for (int step = 0; step < steps; step += 2) {
        const bool two = step + 1 < steps;
        const int base = two ? step * 16 + c * 8 : step * 16 + c * 4;
        uint4 bv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + (g >> 1) * 8 + 2 * j + (g & 1);
          bv[j] = zero;
          if (n < cols && base < rank) {
            const uint16_t* src = b + (int64_t)n * p.R + base;
            if (two) bv[j] = ld_nc(src);
            else {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
              bv[j].x = v.x;
              bv[j].y = v.y;
            }
          }
          if (base + (two ? 8 : 4) > rank) {
            bv[j].x = keep_pair(bv[j].x, base, rank);
            bv[j].y = keep_pair(bv[j].y, base + 2, rank);
            bv[j].z = keep_pair(bv[j].z, base + 4, rank);
            bv[j].w = keep_pair(bv[j].w, base + 6, rank);
          }
        }
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          if (tile0 + m >= tiles) continue;
          const uint4* f = s_frag + ((tile0 + m) * steps + step) * 32 + lane;
#pragma unroll
          for (int term = 0; term < 2; ++term) {
            const uint4 v = f[term * frags];
            const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_bf16_16816(acc[m][j], a, bv[j].x, bv[j].y);
          }
          if (!two) continue;
#pragma unroll
          for (int term = 0; term < 2; ++term) {
            const uint4 v = f[term * frags + 32];
            const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_bf16_16816(acc[m][j], a, bv[j].z, bv[j].w);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!in || row[m][i] < 0) continue;
          uint32_t v[4] = {yv[m][i].x, yv[m][i].y, yv[m][i].z, yv[m][i].w};
          if (rank > 0) {       // (without: the bytes as they are)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[j] = pack_bf16x2(bf16lo_to_f32(v[j]) + acc[m][j][2 * i], bf16hi_to_f32(v[j]) + acc[m][j][2 * i + 1]);
          }
          *reinterpret_cast<uint4*>(out + row[m][i] + col) = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
  }
}

template <int kM>
cudaError_t launch_shrink(const AdapterParams& p, cudaStream_t st) {
  const unsigned grid = (unsigned)p.num_segs * p.groups * p.pieces;
  const int kn = (p.group_ranks + 7) / 8;
  auto go = [&](void (*kernel)(AdapterParams), int n) {
    const size_t smem = (size_t)kAdWarps * kM * 16 * n * 8 * 4;
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return e != cudaSuccess ? e : launch_serialized(kernel, grid, kAdThreads, smem, st, p);
  };
  return kn <= 1   ? go(shrink_kernel<kM, 1>, 1)
         : kn <= 2 ? go(shrink_kernel<kM, 2>, 2)
         : kn <= 4 ? go(shrink_kernel<kM, 4>, 4)
         : kn <= 6 ? go(shrink_kernel<kM, 6>, 6)
                   : go(shrink_kernel<kM, 8>, 8);
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
    // rows of each adapter (the last entry: without one), then their places in the list
    thread_local std::vector<int32_t> count, at;
    thread_local std::vector<AdapterSeg> segs, idle;
    count.assign((size_t)num_adapters + 1, 0);
    int64_t tokens = 0;
    for (int32_t s = 0; s < num_seqs; ++s) {
      if (h_q_len[s] < 0) return internal_failf(HB_ERR_SHAPE, "sequence %d: q_len %d", s, h_q_len[s]);
      if (h_adapter[s] < -1 || h_adapter[s] >= num_adapters)
        return internal_failf(HB_ERR_SHAPE, "sequence %d: adapter %d of %d", s, h_adapter[s], num_adapters);
      tokens += h_q_len[s];
      if (tokens > total_q)
        return internal_failf(HB_ERR_SHAPE, "the sequences have more than total_q (%d) tokens", total_q);
      count[h_adapter[s] < 0 ? num_adapters : h_adapter[s]] += h_q_len[s];
    }
    at.resize(count.size());
    segs.clear();
    idle.clear();
    int32_t run = 0, max_rows = 0;
    for (int32_t a = 0; a <= num_adapters; ++a) {
      at[a] = run;
      // segments of like length, 16-row tiles whole but for the last
      const int32_t n = count[a], pieces = (n + kAdSegRows - 1) / kAdSegRows;
      const int32_t per = pieces ? ((n + pieces - 1) / pieces + 15) / 16 * 16 : 0;
      for (int32_t r = 0; r < n; r += per) {
        const AdapterSeg seg{a < num_adapters ? a : -1, run + r, std::min(per, n - r), 0};
        (a < num_adapters ? segs : idle).push_back(seg);
        if (a < num_adapters) max_rows = std::max(max_rows, seg.rows);
      }
      run += n;
    }
    std::stable_sort(segs.begin(), segs.end(), [](const AdapterSeg& x, const AdapterSeg& y) { return x.rows > y.rows; });
    auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
    AdapterPlan h{};
    h.magic = kAdMagic;
    h.num_seqs = num_seqs;
    h.total_q = total_q;
    h.num_adapters = num_adapters;
    h.max_ranks = max_ranks;
    h.num_sms = num_sms;
    h.num_segs = (int32_t)segs.size();
    h.num_idle_segs = (int32_t)idle.size();
    h.num_rows = run - count[num_adapters];
    h.max_seg_rows = max_rows;
    // pieces of K that fill the SMs twice
    h.max_pieces = segs.empty() ? 1 : std::min<int32_t>(kAdMaxPieces, std::max<int32_t>(1, (2 * num_sms + h.num_segs - 1) / h.num_segs));
    h.ws_rows = (segs.size() + idle.size()) * sizeof(AdapterSeg);
    const uint64_t items = h.ws_rows + (uint64_t)run * 4;
    h.ws_h = up(items);
    h.ws_total = h.ws_h + (uint64_t)h.max_pieces * h.num_rows * max_ranks * 4;
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
    if (!segs.empty()) std::memcpy(body, segs.data(), segs.size() * sizeof(AdapterSeg));
    if (!idle.empty()) std::memcpy(body + segs.size() * sizeof(AdapterSeg), idle.data(), idle.size() * sizeof(AdapterSeg));
    int32_t tok = 0;
    for (int32_t s = 0; s < num_seqs; ++s) {
      int32_t& place = at[h_adapter[s] < 0 ? num_adapters : h_adapter[s]];
      for (int32_t j = 0; j < h_q_len[s]; ++j, ++tok, ++place) std::memcpy(body + h.ws_rows + 4 * (size_t)place, &tok, 4);
    }
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
    int* err = nullptr;
    int num_sms = 0;
    if ((s = internal_device(&err, &num_sms)) != HB_OK) return s;
    uint8_t* ws = static_cast<uint8_t*>(d_workspace);
    AdapterParams p{};
    p.segs = reinterpret_cast<const AdapterSeg*>(ws);
    p.rows = reinterpret_cast<const int32_t*>(ws + h.ws_rows);
    p.num_segs = h.num_segs;
    p.num_rows = h.num_rows;
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
    p.h = reinterpret_cast<float*>(ws + h.ws_h);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (h.num_segs > 0) {
      p.groups = (p.ranks + kAdGroupRanks - 1) / kAdGroupRanks;
      p.group_ranks = ((p.ranks + p.groups - 1) / p.groups + 7) / 8 * 8;
      const int units = (K + 63) / 64;
      const int64_t ctas = (int64_t)h.num_segs * p.groups;
      p.pieces = (int)std::min<int64_t>({h.max_pieces, std::max<int64_t>(1, (2LL * h.num_sms + ctas - 1) / ctas),
                                         std::max(1, units / kAdWarps)});
      p.units_per_piece = (units + p.pieces - 1) / p.pieces;
      p.pieces = (units + p.units_per_piece - 1) / p.units_per_piece;
      if (ctas * p.pieces > 0x7fffffffLL) return internal_fail(HB_ERR_UNSUPPORTED, "too many segments at once");
      const cudaError_t e = h.max_seg_rows <= 16 ? launch_shrink<1>(p, st) : launch_shrink<4>(p, st);
      if (e != cudaSuccess) return internal_failf(HB_ERR_CUDA, "adapter launch: %s", cudaGetErrorString(e));
      internal_note_other_launch(stream);
      internal_count_launch();
    }
    // in place, rows without an adapter have nothing to do
    const int64_t segs = (int64_t)h.num_segs + (in_place ? 0 : h.num_idle_segs);
    if (segs == 0) return internal_ok();
    p.chunk_cols = 8 * kAdWarps * 32;
    int64_t chunks = 0;
    for (;; p.chunk_cols /= 2) {
      chunks = 0;
      for (int i = 0; i < 3; ++i) {
        p.y[i] = static_cast<const uint16_t*>(y->y[i]);
        p.out[i] = static_cast<uint16_t*>(out->y[i]);
        p.cols[i] = y->cols[i];
        p.chunks[i] = (p.cols[i] + p.chunk_cols - 1) / p.chunk_cols;
        chunks += p.chunks[i];
      }
      if (p.chunk_cols == kAdWarps * 32 || segs * chunks >= 4LL * h.num_sms) break;
    }
    if (segs * chunks > 0x7fffffffLL) return internal_fail(HB_ERR_UNSUPPORTED, "too many segments at once");
    const bool small = h.max_seg_rows <= 16 && (in_place || h.num_idle_segs == 0);
    const size_t tiles = (std::max(h.max_seg_rows, 1) + 15) / 16;
    const size_t smem = tiles * ((R + 15) / 16) * 32 * 2 * sizeof(uint4);
    auto kernel = small ? expand_kernel<1> : expand_kernel<2>;
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = launch_serialized(kernel, (unsigned)(segs * chunks), kAdThreads, smem, st, p);
    if (e != cudaSuccess) return internal_failf(HB_ERR_CUDA, "adapter launch: %s", cudaGetErrorString(e));
    internal_note_other_launch(stream);
    internal_count_launch();
    return internal_ok();
  } catch (...) {
    return internal_fail(HB_ERR_CUDA, "unexpected exception in hb_adapters");
  }
}
