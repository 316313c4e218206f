// rope.cu -- rotary positions of a hybrid batch's new tokens, after head norms
// where the model has them, with k and v put into their cache pages (hb_rope),
// and the angles they turn by (hb_rope_phases).
//
// Pair i of a head at position p turns by p f_i: (a, b) becomes (a cos - b sin,
// a sin + b cos) times the attention factor.  p f_i reaches 10^6 radians in long
// contexts, where an fp32 product is off by tenths.  So f_i is held as a
// fraction of a turn in 64-bit fixed point (`phases`): p times it, modulo 2^64,
// is p times the table's value modulo one turn with nothing lost.  Its upper 32
// bits become an fp32 fraction of half a turn (off by 2^-26 of a turn at most,
// whatever the position); the table, computed in 64 bits, is off by less than
// 2^-51 of a turn (2^-54 as measured), which the position multiplies.
//
// Every element is read and written once (k also into its page): HBM bounds
// large batches, launch and latency small ones.  A warp takes one token and some of
// its heads, q's, k's and v's in one list; a lane holds 8 pairs of a head (two
// 16-byte vectors: i and i + rotary_dim / 2 in the half layout, neighbours in the
// interleaved one), which are the same pairs in each of its two to four heads.  The
// warps of a token stand in one CTA, which takes the token's sines and cosines once,
// a thread per pair, in shared memory (each lane taking its own eight: 85.4 us
// instead of 77.8 on the largest case below, 28.0 instead of 24.5 on the one before).
// The rows' loads are issued before the row -> sequence search, as in the append.
//
// Measured on GB300 (a call among others in a graph, inputs not in L2): 68 tokens
// of 8 + 8 heads of 64 2.8 us; 512 of 32 + 8 heads of 128 4.7 us; 2048 of 56 + 8 with
// head norms 22.0 us (3.6 TB/s; the chain of loads, search, angles, sums and stores
// of a token is longer than its bytes); 16205 of 32 + 8 71.4 us (6.0 TB/s, 89 % of
// the copy rate).
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "hb.h"
#include "hb_internal.h"
#include "operands.h"
#include "ptx.cuh"

namespace hb {

hb_status internal_ok();
hb_status internal_check_batch(const hb_batch* b);
hb_status internal_device(int** err, int* num_sms);
void internal_count_launch();
void internal_note_other_launch(void* stream);

namespace {

constexpr int kRopeSmemSeqs = 5500;   // descriptors staged in shared memory up to here (48 KB with the rest)
constexpr int kRopeMaxWarps = 8;      // of a CTA
constexpr int kRopeMaxTokens = 8;

struct RopeParams {
  const int32_t *cu_q_len, *context_len, *block_table;
  int32_t num_seqs, total_q, max_pages_per_seq, num_pages;
  int32_t hq, hkv, heads, chunks;     // heads: q's, k's and (with a cache) v's; chunks: a CTA's warps per token
  int32_t tokens, groups;             // a CTA's tokens (whole, or of one token a group of its warps)
  int32_t rot;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;           // elements between tokens
  uint16_t *q_out, *k_out, *k_cache, *v_cache;    // k_out, caches: or NULL
  int64_t q_out_stride, k_out_stride;
  const uint64_t* phases;
  const uint16_t *q_weight, *k_weight;
  float factor, eps;
  int* dev_error;
};

// Plain loads that leave L1 alone (not .nc: q and k may be written in place).
__device__ __forceinline__ uint4 ld_row(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void widen(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo_to_f32(w[i]);
    f[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}

__device__ __forceinline__ uint4 narrow(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// kIters: heads of a lane; kCtas: CTAs of 8 warps that an SM's registers hold (at least).
template <int D, bool kInterleaved, int kIters, int kCtas>
__global__ void __launch_bounds__(32 * kRopeMaxWarps, kCtas) rope_kernel(const RopeParams p) {
  extern __shared__ int32_t s_cu[];
  __shared__ float2 s_turn[kRopeMaxTokens][D / 2];    // (cos, sin) times the factor
  __shared__ int64_t s_slot[kRopeMaxTokens];          // in the cache, in elements; -1: none, -2: no token
  constexpr int kUnits = D / 16;            // lanes of a head
  constexpr int kHeads = 32 / kUnits;       // heads of a warp at a time
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int mine = warp / p.chunks;         // of the CTA's tokens
  const int tok0 = blockIdx.x / p.groups * p.tokens, tok = tok0 + mine;
  const int unit = lane % kUnits;
  const int head0 = (blockIdx.x % p.groups * p.chunks + warp % p.chunks) * kIters * kHeads + lane / kUnits;
  const bool turns = unit < p.rot / 16;
  // where the lane's two vectors start in a head
  const int at0 = turns && !kInterleaved ? 8 * unit : 16 * unit;
  const int at1 = turns && !kInterleaved ? p.rot / 2 + 8 * unit : 16 * unit + 8;
  auto load = [&](int h, uint4 (&v)[2]) {
    v[0] = v[1] = make_uint4(0, 0, 0, 0);
    if (tok >= p.total_q || h >= p.heads) return;
    const uint16_t* src = h < p.hq           ? p.q + tok * p.q_stride + h * D
                          : h < p.hq + p.hkv ? p.k + tok * p.k_stride + (h - p.hq) * D
                                             : p.v + tok * p.v_stride + (h - p.hq - p.hkv) * D;
    v[0] = ld_row(src + at0);
    v[1] = ld_row(src + at1);
  };
  uint4 in[kIters][2];
#pragma unroll
  for (int it = 0; it < kIters; ++it) load(head0 + it * kHeads, in[it]);
  const bool staged = p.num_seqs <= kRopeSmemSeqs;
  int32_t* s_ctx = s_cu + p.num_seqs + 1;
  if (staged) {
    for (int i = threadIdx.x; i <= p.num_seqs; i += blockDim.x) s_cu[i] = __ldg(&p.cu_q_len[i]);
    for (int i = threadIdx.x; i < p.num_seqs; i += blockDim.x) s_ctx[i] = __ldg(&p.context_len[i]);
  }
  __syncthreads();
  const int32_t* cu = staged ? s_cu : p.cu_q_len;
  const int32_t* ctx = staged ? s_ctx : p.context_len;
  // a thread per pair of a token, and one for its slot
  const int jobs = p.rot / 2 + 1;
  for (int job = threadIdx.x; job < jobs * p.tokens; job += blockDim.x) {
    const int m = job / jobs, i = job % jobs, t = tok0 + m;
    const uint64_t phase = i > 0 ? __ldg(p.phases + i - 1) : 0;
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int q0 = cu[lo], q_len = cu[lo + 1] - q0;
    // (a token of no sequence has no position)
    const bool live = t < p.total_q && (unsigned)(t - q0) < (unsigned)max(q_len, 0);
    const int pos = live ? ctx[lo] - q_len + (t - q0) : -1;
    if (i > 0) {
      // the upper half of position times phase: a signed fraction of half a turn
      float s, c;
      sincospif((float)(int32_t)((phase * (uint64_t)(uint32_t)pos) >> 32) * 0x1p-31f, &s, &c);
      s_turn[m][i - 1] = make_float2(c * p.factor, s * p.factor);
      continue;
    }
    int64_t slot = live ? -1 : -2;
    if (live && pos < 0) {
      report_error(p.dev_error, HB_DEVERR_INDEX);
      slot = -2;
    } else if (live && p.k_cache) {
      const int lp = pos / kPageSize;
      const int page = lp < p.max_pages_per_seq ? __ldg(&p.block_table[(size_t)lo * p.max_pages_per_seq + lp]) : -1;
      if ((unsigned)page < (unsigned)p.num_pages)
        slot = ((int64_t)page * kPageSize + pos % kPageSize) * p.hkv * D;
      else
        report_error(p.dev_error, HB_DEVERR_INDEX);
    }
    s_slot[m] = slot;
  }
  __syncthreads();
  const int64_t slot = s_slot[mine];
  if (slot == -2) return;
  float c[8], s[8];
  if (turns) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 cs = s_turn[mine][8 * unit + e];
      c[e] = cs.x;
      s[e] = cs.y;
    }
  }
  // The head's norm, turn and stores; true (and nothing stored) where its squares leave fp32's range: a sum that
  // overflowed, or one so small that eps does not hide what underflowed.  by: what the head is scaled with before
  // it is squared.
  auto put = [&](int h, const uint4 (&v)[2], float by) {
    const bool is_q = h < p.hq, is_k = !is_q && h < p.hq + p.hkv;
    const uint16_t* w = is_q ? p.q_weight : is_k ? p.k_weight : nullptr;
    float x[16];
    uint4 out[2] = {v[0], v[1]};
    widen(out[0], x);
    widen(out[1], x + 8);
    bool again = false;
    if (p.q_weight || p.k_weight) {       // (all lanes of the warp take part in the sums)
      const float eps = p.eps * by * by;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[e] *= by;
        ss = fmaf(x[e], x[e], ss);
      }
#pragma unroll
      for (int d = kUnits / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      if (w) {
        again = by == 1.f && !(ss <= FLT_MAX && (ss >= 1e-30f || eps >= 1e-30f));
        const float r = rsqrtf(fmaf(ss, 1.f / D, eps));
        float g[16];
        widen(*reinterpret_cast<const uint4*>(w + at0), g);
        widen(*reinterpret_cast<const uint4*>(w + at1), g + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = x[e] * r * g[e];
      }
    }
    if (h >= p.heads || again) return again;
    if (is_q || is_k) {
      if (turns) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float& a = x[kInterleaved ? 2 * e : e];
          float& b = x[kInterleaved ? 2 * e + 1 : 8 + e];
          const float t = a * c[e] - b * s[e];
          b = fmaf(a, s[e], b * c[e]);
          a = t;
        }
      }
      if (turns || w) {
        out[0] = narrow(x);
        out[1] = narrow(x + 8);
      }
    }
    uint16_t* dst = is_q ? p.q_out + tok * p.q_out_stride + h * D
                    : is_k && p.k_out ? p.k_out + tok * p.k_out_stride + (h - p.hq) * D
                                      : nullptr;
    if (dst) {
      *reinterpret_cast<uint4*>(dst + at0) = out[0];
      *reinterpret_cast<uint4*>(dst + at1) = out[1];
    }
    if (!is_q && slot >= 0) {
      dst = is_k ? p.k_cache + slot + (h - p.hq) * D : p.v_cache + slot + (h - p.hq - p.hkv) * D;
      *reinterpret_cast<uint4*>(dst + at0) = out[0];
      *reinterpret_cast<uint4*>(dst + at1) = out[1];
    }
    return false;
  };
  uint32_t rest = 0;    // bit it: the lane's head of that turn is still to be done
#pragma unroll
  for (int it = 0; it < kIters; ++it)
    if (put(head0 + it * kHeads, in[it], 1.f)) rest |= 1u << it;
  // those heads once more, read again (nothing was written in their place) and scaled; rare, and here so that it
  // takes no registers from the others (a sum in 64 bits above: 2048 tokens 29.0 us instead of 22.0)
  if (!__any_sync(0xffffffffu, rest)) return;
#pragma unroll 1
  for (int it = 0; it < kIters; ++it) {
    if (!__any_sync(0xffffffffu, rest >> it & 1)) continue;
    const int h = head0 + it * kHeads;
    const bool there = rest >> it & 1;
    uint4 v[2];
    load(there ? h : p.heads, v);
    float most = 0.f;
    float x[16];
    widen(v[0], x);
    widen(v[1], x + 8);
#pragma unroll
    for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(x[e]));
#pragma unroll
    for (int d = kUnits / 2; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    put(there ? h : p.heads, v, most < 1.f ? 0x1p100f : 0x1p-100f);
  }
}

using RopeKernel = void (*)(RopeParams);
template <int kIters, int kCtas>
RopeKernel rope_kernel_of(int head_dim, bool interleaved) {
  return head_dim == 128 ? (interleaved ? rope_kernel<128, true, kIters, kCtas> : rope_kernel<128, false, kIters, kCtas>)
                         : (interleaved ? rope_kernel<64, true, kIters, kCtas> : rope_kernel<64, false, kIters, kCtas>);
}

}  // namespace
}  // namespace hb

using namespace hb;

extern "C" hb_status hb_rope_phases(int32_t rotary_dim, double base, int32_t scaling, double scale_by,
                                    double original_context, double low, double high, uint64_t* phases) {
  try {
    if (rotary_dim < 16 || rotary_dim % 16)
      return internal_failf(HB_ERR_SHAPE, "rotary_dim %d: a positive multiple of 16 is needed", rotary_dim);
    if (!phases) return internal_fail(HB_ERR_INVALID_ARG, "phases is NULL");
    if (!(base > 1.0 && base <= DBL_MAX)) return internal_failf(HB_ERR_INVALID_ARG, "base %g: must be above 1", base);
    if (scaling < HB_ROPE_PLAIN || scaling > HB_ROPE_PARTS)
      return internal_failf(HB_ERR_INVALID_ARG, "unknown scaling %d", scaling);
    if (scaling != HB_ROPE_PLAIN && !(scale_by >= 1.0 && scale_by <= DBL_MAX))
      return internal_failf(HB_ERR_INVALID_ARG, "scale_by %g: must be at least 1", scale_by);
    if (scaling == HB_ROPE_PARTS &&
        !(original_context > 0 && original_context <= DBL_MAX && low >= 0 && high > low && high <= DBL_MAX))
      return internal_failf(HB_ERR_INVALID_ARG, "parts: original_context %g, low %g, high %g", original_context, low,
                            high);
    const double turn = 6.283185307179586476925;
    const double b = scaling == HB_ROPE_BASE ? base * std::pow(scale_by, rotary_dim / (rotary_dim - 2.0)) : base;
    for (int i = 0; i < rotary_dim / 2; ++i) {
      double f = std::pow(b, -2.0 * i / rotary_dim);
      if (scaling == HB_ROPE_LINEAR) f /= scale_by;
      if (scaling == HB_ROPE_PARTS) {
        const double turns = original_context * f / turn;
        const double keep = std::min(1.0, std::max(0.0, (turns - low) / (high - low)));
        f *= keep + (1.0 - keep) / scale_by;
      }
      phases[i] = (uint64_t)std::ldexp(f / turn, 64);   // (f <= 1: under a sixth of a turn)
    }
    return internal_ok();
  } catch (...) {
    return internal_fail(HB_ERR_CUDA, "unexpected exception in hb_rope_phases");
  }
}

extern "C" hb_status hb_rope(const hb_batch* batch, const hb_rope_params* rope, const void* q, int64_t q_stride,
                             const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* q_out,
                             void* k_out, void* k_cache, void* v_cache, void* stream) {
  try {
    hb_status s = internal_check_batch(batch);
    if (s != HB_OK) return s;
    if (!rope) return internal_fail(HB_ERR_INVALID_ARG, "rope is NULL");
    const int D = batch->head_dim, rot = rope->rotary_dim;
    if (rot < 0 || rot > D || rot % 16)
      return internal_failf(HB_ERR_SHAPE, "rotary_dim %d: a multiple of 16, at most head_dim (%d)", rot, D);
    if (rope->interleaved != 0 && rope->interleaved != 1)
      return internal_failf(HB_ERR_INVALID_ARG, "interleaved %d: 0 or 1", rope->interleaved);
    if (!std::isfinite(rope->factor)) return internal_fail(HB_ERR_INVALID_ARG, "factor must be finite");
    if (!(rope->eps >= 0.f && rope->eps <= FLT_MAX)) return internal_failf(HB_ERR_INVALID_ARG, "eps %g", rope->eps);
    if ((k_cache == nullptr) != (v_cache == nullptr) || (k_cache == nullptr) != (v == nullptr))
      return internal_fail(HB_ERR_INVALID_ARG, "k_cache, v_cache and v go together");
    if (batch->total_q == 0) return internal_ok();
    if (!k_cache && !k_out) return internal_fail(HB_ERR_INVALID_ARG, "k has nowhere to go: neither k_out nor a cache");
    const int64_t T = batch->total_q, qb = 2LL * batch->num_q_heads * D, kb = 2LL * batch->num_kv_heads * D;
    const int64_t pool = (int64_t)batch->num_pages * kPageSize * kb;
    const int64_t qos = q_out == q ? q_stride : qb / 2, kos = k_out == k ? k_stride : kb / 2;
    const Operand in[] = {{q, T, qb, q_stride * 2, "q"},
                          {k, T, kb, k_stride * 2, "k"},
                          {v, T, kb, v_stride * 2, "v"},
                          {rope->q_weight, 1, 2LL * D, 0, "q_weight"},
                          {rope->k_weight, 1, 2LL * D, 0, "k_weight"},
                          {rot ? rope->phases : nullptr, 1, 4LL * rot, 0, "phases"}};
    const Operand out[] = {{q_out, T, qb, qos * 2, "q_out"},
                           {k_out, T, kb, kos * 2, "k_out"},
                           {k_cache, 1, pool, 0, "k_cache"},
                           {v_cache, 1, pool, 0, "v_cache"}};
    for (const Operand& o : in)
      if ((o.p || &o < in + 2 || (rot && &o == in + 5)) && (s = check_rows(o)) != HB_OK) return s;
    for (const Operand& o : out)
      if ((o.p || &o == out) && (s = check_rows(o)) != HB_OK) return s;
    for (int i = 0; i < 4; ++i) {
      for (int j = 0; j < 6; ++j)
        if ((s = check_apart(out[i], in[j], i == j && i < 2)) != HB_OK) return s;
      for (int j = 0; j < i; ++j)
        if ((s = check_apart(out[i], out[j], false)) != HB_OK) return s;
    }
    RopeParams p{};
    int num_sms = 0;
    if ((s = internal_device(&p.dev_error, &num_sms)) != HB_OK) return s;
    p.cu_q_len = batch->cu_q_len;
    p.context_len = batch->context_len;
    p.block_table = batch->block_table;
    p.num_seqs = batch->num_seqs;
    p.total_q = batch->total_q;
    p.max_pages_per_seq = batch->max_pages_per_seq;
    p.num_pages = batch->num_pages;
    p.hq = batch->num_q_heads;
    p.hkv = batch->num_kv_heads;
    p.heads = p.hq + p.hkv * (k_cache ? 2 : 1);
    p.rot = rot;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out = static_cast<uint16_t*>(q_out);
    p.k_out = static_cast<uint16_t*>(k_out);
    p.k_cache = static_cast<uint16_t*>(k_cache);
    p.v_cache = static_cast<uint16_t*>(v_cache);
    p.q_out_stride = qos;
    p.k_out_stride = kos;
    p.phases = rope->phases;
    p.q_weight = static_cast<const uint16_t*>(rope->q_weight);
    p.k_weight = static_cast<const uint16_t*>(rope->k_weight);
    p.factor = rope->factor;
    p.eps = rope->eps;
    // few tokens: two heads per lane, the shortest chain (68 tokens 2.8 us, with four 3.5; 512 4.7 and 4.9); many:
    // four, three CTAs to an SM (16205 tokens 71.4 us; two CTAs 93, three heads 74); with head norms three and four
    // (2048 tokens 22.0 us; four and three 24.8, two and four 23.0; 64 registers spill 22 to 50 bytes).  Between 512
    // and 2048 tokens nothing was measured; below the border head norms go with the few.
    const bool few = T <= 4LL * num_sms, norms = p.q_weight || p.k_weight;
    const int iters = few ? 2 : norms ? 3 : 4;
    const bool inter = rope->interleaved != 0;
    const RopeKernel kernel = few     ? rope_kernel_of<2, 1>(D, inter)
                              : norms ? rope_kernel_of<3, 4>(D, inter)
                                      : rope_kernel_of<4, 3>(D, inter);
    const int per_warp = iters * 32 / (D / 16);
    p.chunks = (p.heads + per_warp - 1) / per_warp;
    // CTAs of whole tokens, up to 8 warps, smaller ones where the tokens are few
    p.groups = (p.chunks + kRopeMaxWarps - 1) / kRopeMaxWarps;
    p.chunks = (p.chunks + p.groups - 1) / p.groups;
    p.tokens = std::min(kRopeMaxTokens, kRopeMaxWarps / p.chunks);
    while (p.tokens > 1 && (T + p.tokens - 1) / p.tokens < 2 * num_sms) p.tokens /= 2;
    const int warps = p.tokens * p.chunks;
    const int64_t grid = (T + p.tokens - 1) / p.tokens * p.groups;
    if (grid > 0x7fffffffLL) return internal_fail(HB_ERR_UNSUPPORTED, "too many tokens and heads at once");
    const size_t smem = p.num_seqs <= kRopeSmemSeqs ? (size_t)(2 * p.num_seqs + 1) * 4 : 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_serialized(kernel, (unsigned)grid, (unsigned)(32 * warps), smem, st, p);
    if (e != cudaSuccess) return internal_failf(HB_ERR_CUDA, "rope launch: %s", cudaGetErrorString(e));
    internal_note_other_launch(stream);
    internal_count_launch();
    return internal_ok();
  } catch (...) {
    return internal_fail(HB_ERR_CUDA, "unexpected exception in hb_rope");
  }
}
