// kv8_widen.cu -- pages of the 8-bit cache spelt out as bf16 in the workspace,
// for the attention of prefill chunks.
//
// A chunk of q tokens reads each cached key q * g / 128 times (once per query
// tile of 128 rows), so its pages are turned into the tensor cores' operand
// type once here instead of once per tile: value * 2^exp is exact in bf16,
// and the attention over the result is the bf16 cache's own (chunk_body.cuh).
// Bytes: one read and two written per element, 3 / (4 q g) of a byte per
// multiply-add that follows.
//
// One CTA takes one page of K or V; a thread turns 16 values (16 bytes) into
// 32 bytes at a time.  The pages go to consecutive places, listed in a block
// table of the workspace's own.
#include <cuda_runtime.h>

#include "hb_internal.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace hb {

namespace {

constexpr int kWidenThreads = 256;

template <int D>
__global__ void __launch_bounds__(kWidenThreads) kv8_widen_kernel(const WidenParams p) {
  const int unit = blockIdx.x >> 1, which = blockIdx.x & 1;
  int lo = 0, hi = p.num_items - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(&p.items[mid].ws_page) <= unit) lo = mid; else hi = mid - 1;
  }
  const WidenItem it = p.items[lo];
  // (hb_kv8_plan writes the items with a copy, which no launch overtakes: they
  // may be read before the wait)
  griddep_wait();
  griddep_launch_dependents();
  const int lp = it.page_begin + unit - it.ws_page;
  const size_t entry = (size_t)it.seq * p.max_pages_per_seq + lp;
  const int page = lp < p.max_pages_per_seq ? __ldcg(&p.block_table[entry]) : -1;
  if ((unsigned)page >= (unsigned)p.num_pages) {
    if (threadIdx.x == 0) {
      report_error(p.dev_error, HB_DEVERR_INDEX);
      if (lp < p.max_pages_per_seq && which == 0) p.ws_table[entry] = -1;
    }
    return;
  }
  if (which == 0 && threadIdx.x == 0) p.ws_table[entry] = unit;
  constexpr int kPerHead = D / 16;   // vectors of 16 values
  const int vecs = kPageSize * p.num_kv_heads * kPerHead;
  const uint4* src = reinterpret_cast<const uint4*>(which ? p.cache[1] : p.cache[0]) + (size_t)page * vecs;
  uint4* dst = reinterpret_cast<uint4*>(which ? p.wide[1] : p.wide[0]) + (size_t)unit * vecs * 2;
  const int8_t* exps = (which ? p.exps[1] : p.exps[0]) + (size_t)page * p.num_kv_heads;
  for (int i = threadIdx.x; i < vecs; i += kWidenThreads) {
    const uint4 v = __ldcg(src + i);
    const float mul = pow2i(kv8_exp(ldcg_s8(exps + (uint32_t)(i / kPerHead) % (uint32_t)p.num_kv_heads)));
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 a = f32x2_of_f16x2(f16x2_of_e4m3x2(in[k]));
      const float2 b = f32x2_of_f16x2(f16x2_of_e4m3x2(in[k] >> 16));
      o[2 * k] = pack_bf16x2(a.x * mul, a.y * mul);
      o[2 * k + 1] = pack_bf16x2(b.x * mul, b.y * mul);
    }
    dst[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace

cudaError_t launch_kv8_widen(const WidenParams& p, cudaStream_t stream) {
  if (p.num_units == 0) return cudaSuccess;
  return launch_serialized(p.head_dim == 128 ? kv8_widen_kernel<128> : kv8_widen_kernel<64>,
                           2u * (unsigned)p.num_units, kWidenThreads, 0, stream, p);
}

}  // namespace hb
