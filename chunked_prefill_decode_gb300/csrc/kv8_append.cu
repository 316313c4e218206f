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
// Where the tokens are fewer than that (decode rows), each token is a unit,
// and those that do not open their page for the batch have nothing to do.
//
// What bounds it: small batches the chain of loads (lengths, table entry, old
// exponent), large ones HBM.  Batches of more pieces than fit the GPU at four
// CTAs per SM take the form with two pieces in flight per warp.  GB300, device
// time per call: 68 tokens (8 heads of 64) 2.5 us; 256 decodes (8 heads of 128)
// 4.9, with page units 7.2; 16201 tokens 20.4 (4.9 TB/s), with one piece per
// warp 39.6.
#include <cuda_runtime.h>

#include <algorithm>

#include "hb.h"
#include "hb_internal.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace hb {

namespace {

constexpr int kA8Threads = 256;
constexpr int kA8CtasPerSm = 2;     // 128 registers a thread: two pieces' rows of 32
constexpr int kA8Warps = kA8Threads / 32;
constexpr int kA8SmemSeqs = 6143;   // cu_q_len and context_len in shared memory up to here (48 KB)

__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// bf16 pair (low half first) times a power of two, as e4m3.
__device__ __forceinline__ uint32_t quantise2(uint32_t v, float mul) {
  float lo, hi;
  unpack_f32x2(mul_f32x2(bf16x2_to_f32x2(v), pack_f32x2(mul, mul)), lo, hi);
  return e4m3x2(lo, hi);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

constexpr uint32_t kInf = 0x7f80u;   // bits of a bf16 infinity; NaN is above

// An element that is not finite as NaN (bits 0x7fff), the others as they are.
__device__ __forceinline__ uint32_t infinite_to_nan2(uint32_t v) {
  if ((v & 0x7fffu) >= kInf) v |= 0x7fffu;
  if (((v >> 16) & 0x7fffu) >= kInf) v |= 0x7fff0000u;
  return v;
}

// |x| bits of a pair, 0 for what is not finite.
__device__ __forceinline__ uint32_t finite_abs2(uint32_t v) {
  uint32_t lo = v & 0x7fffu, hi = (v >> 16) & 0x7fffu;
  lo = lo < kInf ? lo : 0u;
  hi = hi < kInf ? hi : 0u;
  return lo | hi << 16;
}

// One warp's share of the work: the new tokens of one page, one head and one
// of K and V, with their rows on the way to registers.  D bf16 of one token
// and head are D / 8 lanes' 16 bytes, so a warp access covers 256 / D tokens
// and a page takes D / 16 of them.
template <int D>
struct Piece {
  static constexpr int kLanesPerRow = D / 8;
  static constexpr int kRows = 32 / kLanesPerRow;
  static constexpr int kIters = kPageSize / kRows;
  uint4 x[kIters];
  int page;        // block-table entry, checked where it is used
  int part;        // head, or Hkv + head for V; -1: nothing to do
  int old;         // the page's exponent, where it holds older tokens
  int s0, s1;      // slots of the page that receive tokens
};

// Finds the piece and starts its loads (the rows' addresses need no page).
template <int D>
__device__ __forceinline__ void start_piece(const Append8Params& p, const int32_t* cu,
                                            const int32_t* ctxs, uint32_t w, Piece<D>& a) {
  using P = Piece<D>;
  const int lane = threadIdx.x & 31;
  const uint32_t per_unit = 2u * (uint32_t)p.num_kv_heads;
  const uint32_t unit = w / per_unit;
  a.part = -1;
  if (w >= p.num_pieces) return;
  // the sequence whose units hold this one
  int lo = 0, hi = p.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    const uint32_t first = p.by_token ? (uint32_t)cu[mid] : (uint32_t)(cu[mid] >> 4) + 2u * (uint32_t)mid;
    if (first <= unit) lo = mid; else hi = mid - 1;
  }
  const int s = lo;
  const int q0 = cu[s], q_len = cu[s + 1] - q0;
  const int ctx = ctxs[s];
  const int off = ctx - q_len;
  if (q_len <= 0) return;
  if (off < 0 || q0 < 0 || (int64_t)q0 + q_len > p.total_q) {
    if (lane == 0) report_error(p.dev_error, HB_DEVERR_INDEX);
    return;
  }
  int lp;
  if (p.by_token) {
    const uint32_t t = unit - (uint32_t)q0;
    if (t >= (uint32_t)q_len) return;   // a token of no sequence
    lp = (off + (int)t) / kPageSize;
    if (t > 0 && (off + (int)t) % kPageSize) return;
  } else {
    const int k = (int)(unit - (uint32_t)(q0 >> 4) - 2u * (uint32_t)s);
    if (k < 0) return;                  // (before the first sequence's tokens)
    lp = off / kPageSize + k;
  }
  // (lp < ceil(ctx / 16), without adding to a length near 2^31)
  if (lp > (ctx - 1) / kPageSize) return;
  a.page = -1;
  if (lp < p.max_pages_per_seq) a.page = __ldcg(&p.block_table[(size_t)s * p.max_pages_per_seq + lp]);
  // slots s0 .. s1-1 of the page receive tokens tok0 ..
  a.part = (int)(w - unit * per_unit);
  a.s0 = max(0, off - lp * kPageSize);
  a.s1 = min(kPageSize, ctx - lp * kPageSize);
  const int tok0 = q0 + lp * kPageSize + a.s0 - off;
  const bool is_v = a.part >= p.num_kv_heads;
  const int head = is_v ? a.part - p.num_kv_heads : a.part;
  const int sub = lane / P::kLanesPerRow, l = lane % P::kLanesPerRow;
  const size_t row = (size_t)p.num_kv_heads * D;   // elements of one token
  // (where slot `sub` would be; only the slots that receive tokens are read)
  const uint16_t* src = (is_v ? p.v_new : p.k_new) + (int64_t)head * D + l * 8 +
                        ((int64_t)tok0 + sub - a.s0) * (int64_t)row;
#pragma unroll
  for (int i = 0; i < P::kIters; ++i) {
    const uint32_t from = (uint32_t)(i * P::kRows + sub - a.s0);
    a.x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (from < (uint32_t)(a.s1 - a.s0)) a.x[i] = ld_stream16(src + (size_t)(i * P::kRows) * row);
  }
}

template <int D>
__device__ __forceinline__ int8_t* exponent_of(const Append8Params& p, const Piece<D>& a) {
  const bool is_v = a.part >= p.num_kv_heads;
  return (is_v ? p.v_exp : p.k_exp) + (size_t)a.page * p.num_kv_heads +
         (is_v ? a.part - p.num_kv_heads : a.part);
}

// The page is known: checks it, and asks for the exponent that it has.
template <int D>
__device__ __forceinline__ void check_piece(const Append8Params& p, Piece<D>& a) {
  if (a.part < 0) return;
  if ((unsigned)a.page >= (unsigned)p.num_pages) {
    if ((threadIdx.x & 31) == 0) report_error(p.dev_error, HB_DEVERR_INDEX);
    a.part = -1;
    return;
  }
  a.old = kKv8MinExp;
  if (a.s0 > 0) a.old = ldcg_s8(exponent_of(p, a));
}

template <int D>
__device__ __forceinline__ void finish_piece(const Append8Params& p, Piece<D>& a) {
  using P = Piece<D>;
  if (a.part < 0) return;
  const int lane = threadIdx.x & 31;
  const bool is_v = a.part >= p.num_kv_heads;
  const int head = is_v ? a.part - p.num_kv_heads : a.part;
  const int sub = lane / P::kLanesPerRow, l = lane % P::kLanesPerRow;
  const size_t row = (size_t)p.num_kv_heads * D;
  uint8_t* dst = (is_v ? p.v_cache : p.k_cache) +
                 ((size_t)a.page * kPageSize * p.num_kv_heads + head) * D + l * 8;
  const int old = kv8_exp((int8_t)a.old);
  auto largest = [&](auto magnitude) -> uint32_t {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < P::kIters; ++i)
      m = max_u16x2(max_u16x2(m, max_u16x2(magnitude(a.x[i].x), magnitude(a.x[i].y))),
                    max_u16x2(magnitude(a.x[i].z), magnitude(a.x[i].w)));
    return __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  };
  uint32_t m = largest([](uint32_t v) { return v & 0x7fff7fffu; });
  if (m >= kInf) {   // rare: taken over the finite ones instead
    m = largest([](uint32_t v) { return finite_abs2(v); });
#pragma unroll
    for (int i = 0; i < P::kIters; ++i)
      a.x[i] = make_uint4(infinite_to_nan2(a.x[i].x), infinite_to_nan2(a.x[i].y),
                          infinite_to_nan2(a.x[i].z), infinite_to_nan2(a.x[i].w));
  }
  const int e = max(old, kv8_need_exp(m));
  if (e > old && a.s0 > 0) {
    const float down = pow2i(old - e);
    for (int slot = sub; slot < a.s0; slot += P::kRows) {
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
  uint8_t* dst_sub = dst + (size_t)sub * row;
#pragma unroll
  for (int i = 0; i < P::kIters; ++i) {
    if (i * P::kRows >= a.s1 || (i + 1) * P::kRows <= a.s0) continue;   // (alike in the warp)
    if ((uint32_t)(i * P::kRows + sub - a.s0) < (uint32_t)(a.s1 - a.s0))
      *reinterpret_cast<uint2*>(dst_sub + (size_t)(i * P::kRows) * row) =
          make_uint2(quantise2(a.x[i].x, mul) | quantise2(a.x[i].y, mul) << 16,
                     quantise2(a.x[i].z, mul) | quantise2(a.x[i].w, mul) << 16);
  }
  __syncwarp();   // every lane has read the old exponent
  if (lane == 0) *exponent_of(p, a) = (int8_t)e;
}

// kMany: each warp takes pieces w, w + warps, .. and starts the next one's
// loads before it finishes the one at hand; else one piece per warp, in more
// and smaller warps.
template <int D, bool kMany>
__global__ void __launch_bounds__(kA8Threads, kMany ? kA8CtasPerSm : 4)
    kv8_append_kernel(const Append8Params p) {
  extern __shared__ int32_t s_cu[];
  griddep_wait();
  griddep_launch_dependents();
  const bool staged = p.num_seqs <= kA8SmemSeqs;
  int32_t* s_ctx = s_cu + p.num_seqs + 1;
  if (staged) {
    for (int i = threadIdx.x; i <= p.num_seqs; i += kA8Threads) s_cu[i] = __ldcg(&p.cu_q_len[i]);
    for (int i = threadIdx.x; i < p.num_seqs; i += kA8Threads) s_ctx[i] = __ldcg(&p.context_len[i]);
  }
  __syncthreads();
  const int32_t* cu = staged ? s_cu : p.cu_q_len;
  const int32_t* ctxs = staged ? s_ctx : p.context_len;
  uint32_t w = blockIdx.x * kA8Warps + (threadIdx.x >> 5);
  Piece<D> a;
  start_piece<D>(p, cu, ctxs, w, a);
  check_piece<D>(p, a);
  if constexpr (!kMany) {
    finish_piece<D>(p, a);
  } else {
    // (two pieces by name: a copy would wait for the loads)
    const uint32_t step = gridDim.x * kA8Warps;
    Piece<D> b;
    for (; w < p.num_pieces; w += 2 * step) {
      start_piece<D>(p, cu, ctxs, w + step, b);
      finish_piece<D>(p, a);
      check_piece<D>(p, b);
      start_piece<D>(p, cu, ctxs, w + 2 * step, a);
      finish_piece<D>(p, b);
      check_piece<D>(p, a);
    }
  }
}

}  // namespace

cudaError_t launch_kv8_append(Append8Params p, int head_dim, int num_sms, cudaStream_t stream) {
  const int64_t pieces = kv8_append_pieces(p.total_q, p.num_seqs, p.num_kv_heads);
  if (pieces > 0x7fffffffLL) return cudaErrorInvalidValue;   // (w + step stays within 32 bits)
  p.num_pieces = (uint32_t)pieces;
  p.by_token = kv8_append_by_token(p.total_q, p.num_seqs);
  int64_t blocks = (pieces + kA8Warps - 1) / kA8Warps;
  const bool many = blocks > 4 * 2LL * num_sms;
  if (many) blocks = (int64_t)kA8CtasPerSm * num_sms;
  const size_t smem = p.num_seqs <= kA8SmemSeqs ? (size_t)(2 * p.num_seqs + 1) * 4 : 0;
  const auto kernel = head_dim == 128 ? (many ? kv8_append_kernel<128, true> : kv8_append_kernel<128, false>)
                                      : (many ? kv8_append_kernel<64, true> : kv8_append_kernel<64, false>);
  return launch_serialized(kernel, (unsigned)blocks, kA8Threads, smem, stream, p);
}

}  // namespace hb
