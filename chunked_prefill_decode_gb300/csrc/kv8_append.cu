// kv8_append.cu -- the batch's new K/V rows quantised into the 8-bit cache.
//
// Same place in a step as kv_append.cu ("Sarathi-Serve：以 chunked-prefills 与
// stall-free batching 驯服 LLM 推理的吞吐—延迟权衡", §GPU / 系统数据路径 ⑤), into
// pages of e4m3 values with one exponent per (page, kv head) (kv8.cuh):
//   need(x) = the smallest e with max |x| <= 448 * 2^e over the page's new
//             finite values of that head,
//   e       = need on a page that the batch starts, max(old e, need) on one
//             that holds older tokens (whose values, should e grow, become
//             round(value * 2^(old e - e))),
//   value   = round_e4m3(x * 2^-e); infinities and NaN become NaN, since the
//             format has no infinity and a large finite value would hide it.
//
// The scale belongs to a page and head, so that is the unit of work: one warp
// takes all the new tokens (1 to 16) of one page, one kv head and one of K
// and V, holds them in registers between the maximum and the rounding, and
// nothing is read twice.  Bytes: 2 T Hkv D * 2 read, half of that written.
//
// Which page a warp works on follows from cu_q_len alone: sequence s has the
// units floor(cu[s] / 16) + 2 s and up, floor(cu[s+1] / 16) - floor(cu[s] / 16)
// + 2 of them, which is never less than the pages that its tokens touch; a
// warp that draws a unit past them has nothing to do.  So the grid is known
// on the host (total_q / 16 + 2 num_seqs units) and the device needs no
// prefix sum over pages, only the search in cu_q_len that every append makes.
#include <cuda_runtime.h>

#include <algorithm>

#include "hb.h"
#include "hb_internal.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace hb {

namespace {

constexpr int kA8Threads = 256;
constexpr int kA8Warps = kA8Threads / 32;
constexpr int kA8SmemSeqs = 6143;   // cu_q_len and context_len in shared memory up to here (48 KB)

__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// bf16 pair (low half first) times a power of two, as e4m3; an infinity
// becomes NaN.
__device__ __forceinline__ uint32_t quantise2(uint32_t v, float mul) {
  float lo = bf16lo_to_f32(v), hi = bf16hi_to_f32(v);
  if ((v & 0x7fffu) == 0x7f80u) lo = __uint_as_float(0x7fc00000u);
  if ((v & 0x7fff0000u) == 0x7f800000u) hi = __uint_as_float(0x7fc00000u);
  return e4m3x2(lo * mul, hi * mul);
}

// the largest |x| (as bits) of the finite values of a pair
__device__ __forceinline__ uint32_t finite_max2(uint32_t v) {
  uint32_t lo = v & 0x7fffu, hi = (v >> 16) & 0x7fffu;
  lo = lo < 0x7f80u ? lo : 0u;
  hi = hi < 0x7f80u ? hi : 0u;
  return max(lo, hi);
}

// D bf16 of one token and head are D / 8 lanes' 16 bytes, so a warp access
// covers kRows tokens and a page takes 16 / kRows of them.
template <int D>
__global__ void __launch_bounds__(kA8Threads) kv8_append_kernel(const Append8Params p) {
  constexpr int kLanesPerRow = D / 8;
  constexpr int kRows = 32 / kLanesPerRow;
  constexpr int kIters = kPageSize / kRows;
  extern __shared__ int32_t s_cu[];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const bool staged = p.num_seqs <= kA8SmemSeqs;
  int32_t* s_ctx = s_cu + p.num_seqs + 1;
  if (staged) {
    for (int i = threadIdx.x; i <= p.num_seqs; i += kA8Threads) s_cu[i] = __ldcg(&p.cu_q_len[i]);
    for (int i = threadIdx.x; i < p.num_seqs; i += kA8Threads) s_ctx[i] = __ldcg(&p.context_len[i]);
  }
  __syncthreads();
  const int32_t* cu = staged ? s_cu : p.cu_q_len;
  const int32_t* ctxs = staged ? s_ctx : p.context_len;

  const int64_t w = (int64_t)blockIdx.x * kA8Warps + (threadIdx.x >> 5);
  const int per_unit = 2 * p.num_kv_heads;
  const int64_t unit = w / per_unit;
  const int part = (int)(w - unit * per_unit);
  const bool is_v = part >= p.num_kv_heads;
  const int head = is_v ? part - p.num_kv_heads : part;
  if (unit >= p.num_units) return;
  // the sequence whose units hold this one
  int lo = 0, hi = p.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((cu[mid] >> 4) + 2 * (int64_t)mid <= unit) lo = mid; else hi = mid - 1;
  }
  const int s = lo;
  const int q0 = cu[s], q_len = cu[s + 1] - q0;
  const int ctx = ctxs[s];
  const int off = ctx - q_len;
  const int k = (int)(unit - (q0 >> 4) - 2 * (int64_t)s);
  if (q_len <= 0) return;
  if (off < 0 || q0 < 0 || q0 + q_len > p.total_q) {
    if (lane == 0) report_error(p.dev_error, HB_DEVERR_INDEX);
    return;
  }
  const int lp = off / kPageSize + k;
  // (lp < ceil(ctx / 16), without adding to a length near 2^31)
  if (lp > (ctx - 1) / kPageSize) return;
  int page = -1;
  if (lp < p.max_pages_per_seq) page = __ldcg(&p.block_table[(size_t)s * p.max_pages_per_seq + lp]);
  if ((unsigned)page >= (unsigned)p.num_pages) {
    if (lane == 0) report_error(p.dev_error, HB_DEVERR_INDEX);
    return;
  }
  // slots s0 .. s1-1 of the page receive tokens tok0 ..
  const int s0 = max(0, off - lp * kPageSize);
  const int s1 = min(kPageSize, ctx - lp * kPageSize);
  const int tok0 = q0 + lp * kPageSize + s0 - off;
  const int sub = lane / kLanesPerRow, l = lane % kLanesPerRow;
  const uint16_t* src = is_v ? p.v_new : p.k_new;
  const size_t row = (size_t)p.num_kv_heads * D;   // elements of one token
  src += ((size_t)tok0 * p.num_kv_heads + head) * D + l * 8;
  uint4 x[kIters];
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int slot = i * kRows + sub;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= s0 && slot < s1) x[i] = ld_stream16(src + (size_t)(slot - s0) * row);
  }
  int8_t* exps = (is_v ? p.v_exp : p.k_exp) + (size_t)page * p.num_kv_heads + head;
  uint8_t* dst = (is_v ? p.v_cache : p.k_cache) + ((size_t)page * kPageSize * p.num_kv_heads + head) * D + l * 8;
  const int old = s0 > 0 ? kv8_exp(ldcg_s8(exps)) : kKv8MinExp;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kIters; ++i)
    m = max(max(m, max(finite_max2(x[i].x), finite_max2(x[i].y))),
            max(finite_max2(x[i].z), finite_max2(x[i].w)));
  m = __reduce_max_sync(0xffffffffu, m);
  const int e = max(old, kv8_need_exp(m));
  if (s0 > 0 && e > old) {
    const float down = pow2i(old - e);
    for (int slot = sub; slot < s0; slot += kRows) {
      uint2 v = *reinterpret_cast<const uint2*>(dst + (size_t)slot * row);
      uint32_t* b = &v.x;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 f0 = f32x2_of_f16x2(f16x2_of_e4m3x2(b[h]));
        const float2 f1 = f32x2_of_f16x2(f16x2_of_e4m3x2(b[h] >> 16));
        b[h] = e4m3x2(f0.x * down, f0.y * down) | e4m3x2(f1.x * down, f1.y * down) << 16;
      }
      *reinterpret_cast<uint2*>(dst + (size_t)slot * row) = v;
    }
  }
  const float mul = pow2i(-e);
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int slot = i * kRows + sub;
    if (slot >= s0 && slot < s1)
      *reinterpret_cast<uint2*>(dst + (size_t)slot * row) =
          make_uint2(quantise2(x[i].x, mul) | quantise2(x[i].y, mul) << 16,
                     quantise2(x[i].z, mul) | quantise2(x[i].w, mul) << 16);
  }
  __syncwarp();   // every lane has read the old exponent
  if (lane == 0) *exps = (int8_t)e;
}

}  // namespace

cudaError_t launch_kv8_append(Append8Params p, int head_dim, cudaStream_t stream) {
  p.num_units = p.total_q / kPageSize + 2LL * p.num_seqs;
  const int64_t warps = p.num_units * 2 * p.num_kv_heads;
  const int64_t blocks = (warps + kA8Warps - 1) / kA8Warps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const size_t smem = p.num_seqs <= kA8SmemSeqs ? (size_t)(2 * p.num_seqs + 1) * 4 : 0;
  return launch_serialized(head_dim == 128 ? kv8_append_kernel<128> : kv8_append_kernel<64>,
                           (unsigned)blocks, kA8Threads, smem, stream, p);
}

}  // namespace hb
