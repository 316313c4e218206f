// attention8.cu -- the attention launch over the 8-bit cache (kv8.cuh).
//
// As attention.cu: one grid, decode CTAs first (decode8_body.cuh, streaming
// the 8-bit pages as they are), then one CTA per chunk item (chunk_body.cuh,
// over the chunk rows' pages that kv8_widen.cu has spelt out as bf16 in the
// launch before).  The decode CTAs do not wait for that launch, only for the
// append, so they stream while the pages are widened.
#include <cuda_runtime.h>

#include <atomic>

#include "chunk_body.cuh"
#include "decode8_body.cuh"
#include "hb_internal.h"
#include "ptx.cuh"

namespace hb {

constexpr int kAttn8Threads = 384;

struct Attn8Params {
  DecodeParams dec;
  Decode8Params dec8;
  Decode8Layout dl;
  ChunkParams chk;
  int32_t decode_grid;
  // 1: the launch before this one let it start with everything complete but
  // its own results: the append's (the decode CTAs wait before the pages with
  // new tokens, dec8.wait_new), or the widened pages (the chunk CTAs wait
  // before they read one, chk.wait_first)
  int32_t early;
};

template <int D, bool kPairs, bool kFew>
__global__ void __launch_bounds__(kAttn8Threads, 1)
    attention8_kernel(const Attn8Params p, const __grid_constant__ CUtensorMap dec_k,
                      const __grid_constant__ CUtensorMap dec_v,
                      const __grid_constant__ CUtensorMap chunk_q,
                      const __grid_constant__ CUtensorMap chunk_k,
                      const __grid_constant__ CUtensorMap chunk_v) {
  extern __shared__ uint8_t smem_raw[];
  if (!p.early) griddep_wait();
  griddep_launch_dependents();
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  if ((int)blockIdx.x < p.decode_grid)
    decode8_cta<D>(p.dec, p.dec8, p.dl, dec_k, dec_v, smem, blockIdx.x);
  else
    chunk_cta<D, kPairs, kFew>(p.chk, chunk_q, chunk_k, chunk_v, chunk_k, chunk_v, nullptr, nullptr,
                               smem, blockIdx.x - p.decode_grid);
}

// As launch_attention (attention.cu): decode_grid decode CTAs, then one CTA
// per chunk item, either part possibly empty; pairs_mode as there; device:
// the current one (below 64).
cudaError_t launch_attention8(const DecodeParams& dec, const Decode8Params& dec8, int decode_grid,
                              const ChunkParams& chk, int head_dim, const CUtensorMap& dec_k,
                              const CUtensorMap& dec_v, const CUtensorMap& chunk_q,
                              const CUtensorMap& chunk_k, const CUtensorMap& chunk_v,
                              cudaStream_t stream, bool early, int pairs_mode, int device) {
  Attn8Params p{};
  p.early = early ? 1 : 0;
  p.dec = dec;
  p.dec8 = dec8;
  p.chk = chk;
  p.decode_grid = dec.num_items > 0 ? decode_grid : 0;
  p.dl = decode8_layout(head_dim, dec.kvh_block, dec.group);
  if (p.decode_grid > 0 && p.dl.n_stages < 2) return cudaErrorInvalidConfiguration;
  const int grid = p.decode_grid + chk.num_items;
  if (grid == 0) return cudaSuccess;
  const int chunk_smem = head_dim == 128 ? ChunkCfg<128>::kSmemBytes : ChunkCfg<64>::kSmemBytes;
  const int smem = p.dl.smem_bytes > chunk_smem ? p.dl.smem_bytes : chunk_smem;
  using Kernel = void (*)(const Attn8Params, const __grid_constant__ CUtensorMap,
                          const __grid_constant__ CUtensorMap, const __grid_constant__ CUtensorMap,
                          const __grid_constant__ CUtensorMap, const __grid_constant__ CUtensorMap);
  if (pairs_mode < 0 || pairs_mode > 3) return cudaErrorInvalidValue;
  const int which = (head_dim == 128 ? 4 : 0) + pairs_mode;
  const Kernel kernels[8] = {attention8_kernel<64, false, false>,  attention8_kernel<64, true, false>,
                             attention8_kernel<64, false, true>,   attention8_kernel<64, true, true>,
                             attention8_kernel<128, false, false>, attention8_kernel<128, true, false>,
                             attention8_kernel<128, false, true>,  attention8_kernel<128, true, true>};
  const Kernel kernel = kernels[which];
  // the chunk CTAs' register split assumes kChunkLaunchRegs per thread at
  // launch (attention.cu)
  static std::atomic<int> regs[8] = {};
  int n = regs[which].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaFuncAttributes fa{};
    const cudaError_t ea = cudaFuncGetAttributes(&fa, kernel);
    if (ea != cudaSuccess) return ea;
    n = fa.numRegs;
    regs[which].store(n, std::memory_order_relaxed);
  }
  if (n < kChunkLaunchRegs) return cudaErrorInvalidConfiguration;
  // (the opt-in to the largest shared memory holds for a device once made)
  static std::atomic<uint64_t> opted[8] = {};
  const uint64_t bit = 1ull << device;
  if (!(opted[which].load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    opted[which].fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_serialized(kernel, grid, kAttn8Threads, smem, stream, p, dec_k, dec_v, chunk_q, chunk_k,
                           chunk_v);
}

}  // namespace hb
