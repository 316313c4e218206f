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
// exponent), large ones HBM.  Batches of more than eight CTAs per SM of single
// pieces (K and V apart; four are resident, so two rounds of them) take the
// form where a warp keeps K and V of a page in flight and finds the place of
// both at once (with a place for each, 661 instructions a piece and half the
// issue slots).  GB300, device time per call: 68 tokens (8
// heads of 64) 2.6 us; 256 decodes (8 heads of 128) 4.8, with page units 7.2;
// 16201 tokens from HBM 20.8 (4.8 TB/s), from L2 15.2, with a place for each
// 23.9 and 20.5, with one piece per warp 39.6 from L2.
#include <cuda_runtime.h>

#include <algorithm>

#include "hb.h"
#include "hb_internal.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace hb {

namespace {

constexpr int kA8Threads = 256;
// CTAs per SM of the form for large batches: K's and V's rows of a page take 64
// registers a thread at D 128, 32 at D 64 (16 x 2021 tokens of 8 heads: 20.3
// us, with three CTAs 20.8, with two 23.6).
constexpr int a8_ctas_per_sm(int head_dim) { return head_dim == 128 ? 2 : 4; }
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

// The new tokens of one page and one head, K or V or both.  D bf16 of one
// token and head are D / 8 lanes' 16 bytes, so a warp access covers 256 / D
// tokens and a page takes D / 16 of them (kIters).
template <int D>
struct Rows {
  static constexpr int kLanesPerRow = D / 8;
  static constexpr int kRows = 32 / kLanesPerRow;
  static constexpr int kIters = kPageSize / kRows;
};

struct Place {
  int page;        // block-table entry, checked where it is used
  int head;        // -1: nothing to do
  int s0, s1;      // slots of the page that receive tokens
  int tok;         // the token that slot 0 holds, or would (below 0 at worst by 15)
};

// Finds the place of unit `unit`; the table entry may still be on its way.
__device__ __forceinline__ Place find_place(const Append8Params& p, const int32_t* cu,
                                            const int32_t* ctxs, uint32_t unit, int head) {
  Place a;
  a.page = a.head = -1;
  a.s0 = a.s1 = a.tok = 0;
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
  if (q_len <= 0) return a;
  if (off < 0 || q0 < 0 || (int64_t)q0 + q_len > p.total_q) {
    if ((threadIdx.x & 31) == 0) report_error(p.dev_error, HB_DEVERR_INDEX);
    return a;
  }
  int lp;
  if (p.by_token) {
    const uint32_t t = unit - (uint32_t)q0;
    if (t >= (uint32_t)q_len) return a;   // a token of no sequence
    lp = (off + (int)t) / kPageSize;
    if (t > 0 && (off + (int)t) % kPageSize) return a;
  } else {
    const int k = (int)(unit - (uint32_t)(q0 >> 4) - 2u * (uint32_t)s);
    if (k < 0) return a;                  // (before the first sequence's tokens)
    lp = off / kPageSize + k;
  }
  // (lp < ceil(ctx / 16), without adding to a length near 2^31)
  if (lp > (ctx - 1) / kPageSize) return a;
  if (lp < p.max_pages_per_seq) a.page = __ldcg(&p.block_table[(size_t)s * p.max_pages_per_seq + lp]);
  a.head = head;
  a.s0 = max(0, off - lp * kPageSize);
  a.s1 = min(kPageSize, ctx - lp * kPageSize);
  a.tok = q0 + (lp * kPageSize - off);
  return a;
}

// Starts the loads of its rows of `src` (k_new or v_new; no page is needed).
template <int D>
__device__ __forceinline__ void load_rows(const Append8Params& p, const Place& a, const uint16_t* src,
                                          uint4* x) {
  using R = Rows<D>;
  if (a.head < 0) return;
  const int lane = threadIdx.x & 31, sub = lane / R::kLanesPerRow, l = lane % R::kLanesPerRow;
  const size_t row = (size_t)p.num_kv_heads * D;   // elements of one token
  // (only the slots that receive tokens are read)
  const uint16_t* at = src + (int64_t)a.head * D + l * 8 + ((int64_t)a.tok + sub) * (int64_t)row;
  if (a.s1 - a.s0 == kPageSize) {
#pragma unroll
    for (int i = 0; i < R::kIters; ++i) x[i] = ld_stream16(at + (size_t)(i * R::kRows) * row);
  } else {
#pragma unroll
    for (int i = 0; i < R::kIters; ++i) {
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if ((uint32_t)(i * R::kRows + sub - a.s0) < (uint32_t)(a.s1 - a.s0))
        x[i] = ld_stream16(at + (size_t)(i * R::kRows) * row);
    }
  }
}

// The page is known: false (and reported) if it is none.
__device__ __forceinline__ bool check_page(const Append8Params& p, const Place& a) {
  if (a.head < 0) return false;
  if ((unsigned)a.page < (unsigned)p.num_pages) return true;
  if ((threadIdx.x & 31) == 0) report_error(p.dev_error, HB_DEVERR_INDEX);
  return false;
}

// Quantises the rows into `cache` (k_cache or v_cache), with `exps` its
// exponents.
template <int D>
__device__ __forceinline__ void finish_rows(const Append8Params& p, const Place& a, uint8_t* cache,
                                            int8_t* exps, uint4* x) {
  using R = Rows<D>;
  const int lane = threadIdx.x & 31, sub = lane / R::kLanesPerRow, l = lane % R::kLanesPerRow;
  const size_t row = (size_t)p.num_kv_heads * D;
  uint8_t* dst = cache + ((size_t)a.page * kPageSize * p.num_kv_heads + a.head) * D + l * 8;
  int8_t* exp_at = exps + (size_t)a.page * p.num_kv_heads + a.head;
  const int old = a.s0 > 0 ? kv8_exp(ldcg_s8(exp_at)) : kKv8MinExp;
  auto largest = [&](auto magnitude) -> uint32_t {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < R::kIters; ++i)
      m = max_u16x2(max_u16x2(m, max_u16x2(magnitude(x[i].x), magnitude(x[i].y))),
                    max_u16x2(magnitude(x[i].z), magnitude(x[i].w)));
    return __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  };
  uint32_t m = largest([](uint32_t v) { return v & 0x7fff7fffu; });
  if (m >= kInf) {   // rare: taken over the finite ones instead
    m = largest([](uint32_t v) { return finite_abs2(v); });
#pragma unroll
    for (int i = 0; i < R::kIters; ++i)
      x[i] = make_uint4(infinite_to_nan2(x[i].x), infinite_to_nan2(x[i].y), infinite_to_nan2(x[i].z),
                        infinite_to_nan2(x[i].w));
  }
  const int e = max(old, kv8_need_exp(m));
  if (e > old && a.s0 > 0) {
    const float down = pow2i(old - e);
    for (int slot = sub; slot < a.s0; slot += R::kRows) {
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
  auto quantised = [&](const uint4& v) {
    return make_uint2(quantise2(v.x, mul) | quantise2(v.y, mul) << 16,
                      quantise2(v.z, mul) | quantise2(v.w, mul) << 16);
  };
  if (a.s1 - a.s0 == kPageSize) {
#pragma unroll
    for (int i = 0; i < R::kIters; ++i)
      *reinterpret_cast<uint2*>(dst_sub + (size_t)(i * R::kRows) * row) = quantised(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < R::kIters; ++i) {
      if (i * R::kRows >= a.s1 || (i + 1) * R::kRows <= a.s0) continue;   // (alike in the warp)
      if ((uint32_t)(i * R::kRows + sub - a.s0) < (uint32_t)(a.s1 - a.s0))
        *reinterpret_cast<uint2*>(dst_sub + (size_t)(i * R::kRows) * row) = quantised(x[i]);
    }
  }
  __syncwarp();   // every lane has read the old exponent
  if (lane == 0) *exp_at = (int8_t)e;
}

// kMany: a warp takes K and V of a page and head at once (their places, rows
// and checks are alike), w, w + warps, .., and starts the next ones' loads as
// it finishes those at hand; else K or V, one per warp, in more and smaller
// warps.
template <int D, bool kMany>
__global__ void __launch_bounds__(kA8Threads, kMany ? a8_ctas_per_sm(D) : 4)
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
  const uint32_t heads = (uint32_t)p.num_kv_heads;
  uint32_t w = blockIdx.x * kA8Warps + (threadIdx.x >> 5);
  if constexpr (!kMany) {
    if (w >= p.num_pieces) return;
    const uint32_t unit = w / (2u * heads), part = w - unit * 2u * heads;
    const bool is_v = part >= heads;
    const Place a = find_place(p, cu, ctxs, unit, (int)(is_v ? part - heads : part));
    uint4 x[Rows<D>::kIters];
    load_rows<D>(p, a, is_v ? p.v_new : p.k_new, x);
    if (check_page(p, a)) finish_rows<D>(p, a, is_v ? p.v_cache : p.k_cache, is_v ? p.v_exp : p.k_exp, x);
  } else {
    const uint32_t step = gridDim.x * kA8Warps, pairs = p.num_pieces / 2u;
    uint4 xk[Rows<D>::kIters], xv[Rows<D>::kIters];
    auto place = [&](uint32_t i) -> Place {
      const uint32_t unit = i / heads;
      if (i < pairs) return find_place(p, cu, ctxs, unit, (int)(i - unit * heads));
      return Place{-1, -1, 0, 0, 0};
    };
    Place a = place(w);
    load_rows<D>(p, a, p.k_new, xk);
    load_rows<D>(p, a, p.v_new, xv);
    for (; w < pairs; w += step) {
      const Place b = place(w + step);
      const bool ok = check_page(p, a);
      if (ok) finish_rows<D>(p, a, p.k_cache, p.k_exp, xk);
      load_rows<D>(p, b, p.k_new, xk);
      if (ok) finish_rows<D>(p, a, p.v_cache, p.v_exp, xv);
      load_rows<D>(p, b, p.v_new, xv);
      a = b;
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
  const bool many = blocks > 8LL * num_sms;   // (see above)
  if (many) blocks = std::min<int64_t>((blocks + 1) / 2, (int64_t)a8_ctas_per_sm(head_dim) * num_sms);
  const size_t smem = p.num_seqs <= kA8SmemSeqs ? (size_t)(2 * p.num_seqs + 1) * 4 : 0;
  const auto kernel = head_dim == 128 ? (many ? kv8_append_kernel<128, true> : kv8_append_kernel<128, false>)
                                      : (many ? kv8_append_kernel<64, true> : kv8_append_kernel<64, false>);
  return launch_serialized(kernel, (unsigned)blocks, kA8Threads, smem, stream, p);
}

}  // namespace hb
