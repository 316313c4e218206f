// norm.cu -- the norm after a branch of a transformer block, its gate and
// residual scale, the residual sum and the norm before the next branch, in one
// pass over the rows of the residual stream (hb_norm).
//
//   u  = y * rsqrt(mean(y^2) + eps) * (offset + w_post)      (w_post given)
//   x' = residual_scale * x + branch_scale * gate * u
//   z  = x' * rsqrt(mean(x'^2) + eps) * (offset + w_pre)
//
// Each element is read and written once, and a dozen operations are done on
// it, so HBM bounds it (launch and latency where the rows are few).  A row
// belongs to a group of threads that hold it in registers as fp32 from the
// load to the last store, so that z is the norm of the sum before its rounding
// and no operand is read twice; the two means are sums over a warp's lanes and
// then, through shared memory, over the group's warps, in a fixed order.
//
// Measured on GB300 (a call among others in a graph, inputs not in L2): one row of
// 7168 2.5 us; 512 rows of 4096, sum and norm, 5.1 us (3.3 TB/s); 2048 of 7168, both
// norms, fp32 stream, 37.9 us (4.6 TB/s, 69 % of the copy rate); 8191 of 4096, both
// norms, gates per row, 59.6 us (5.6 TB/s, 83 %).  Two or four vectors per thread
// instead of one where rows are many: 65.7 us against 78 for the last one (fewer
// warps to a row's sums).  Rows kept packed until used and weights loaded late, for
// 85 registers and a third CTA on the SM: 39.3 us against 37.9 on 2048 rows (it spills;
// so do, at 128 registers, four vectors of an fp32 stream, 84 bytes, of a bf16 one, 52,
// and the kernel of many rows, 56).
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "hb.h"
#include "hb_internal.h"
#include "operands.h"
#include "ptx.cuh"
#include "ring.h"

namespace hb {

hb_status internal_ok();
hb_status internal_device(int** err, int* num_sms);
void internal_count_launch();
void internal_note_other_launch(void* stream);

namespace {

// threads of a row (at most) where each holds `per` vectors: what its
// registers allow
__host__ __device__ constexpr int norm_max_threads(int per) { return per == 1 ? 1024 : 512; }
constexpr int kNormMaxWidth = 8 * 4 * norm_max_threads(4);

struct NormParams {
  int32_t rows, vecs;                 // vecs: 8-element vectors of a row
  int32_t threads_per_row;            // a multiple of 32
  const uint16_t *y, *gate, *w_post, *w_pre;
  const void* x;                      // bf16 or fp32
  void* x_out;
  uint16_t* z;
  int64_t x_stride, y_stride, gate_stride, x_out_stride, z_stride;   // elements
  float eps, residual_scale, branch_scale, offset, inv_width;
  int* dev_error;
};

__device__ __forceinline__ void widen8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo_to_f32(w[i]);
    f[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}

__device__ __forceinline__ uint4 narrow8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Sum over the row's threads (all of them get it).  `part`: the row's slots,
// one per warp, used once.
template <typename T>
__device__ __forceinline__ T row_sum(T v, T* part, int warps, int bar) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % warps;
  if (lane == 0) part[warp] = v;
  named_bar_sync(bar, warps * 32);
  if (warps <= 8) {
    v = part[0];
#pragma unroll
    for (int w = 1; w < 8; ++w)
      if (w < warps) v += part[w];
    return v;
  }
  v = lane < warps ? part[lane] : T(0);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// rsqrt(mean of squares + eps) of the row.  Squares that leave fp32's range (a
// sum that overflowed, or one so small that eps does not hide what
// underflowed) are summed again in 64 bits: rare, and the same for all threads
// of the row.
// kNoEps (eps is 0, the only one that lets a root fall below 2^-100, where fp32 may not
// hold its inverse): such a row is scaled by 2^64, f here and `stage`, where f was read
// from and is read from again (this thread's vectors of a staged row, blockDim.x
// apart; or NULL).  Other calls do without: 62.4 us instead of 60.4 on 8191 gated rows of 4096.
template <int kVecs, bool kNoEps>
__device__ __forceinline__ float row_scale(float (&f)[kVecs][8], float* part, double* wide, int warps, int bar,
                                           const NormParams& p, uint4* stage = nullptr) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(f[i][e], f[i][e], ss);
  ss = row_sum(ss, part, warps, bar);
  if (ss <= FLT_MAX && (ss >= 1e-30f || p.eps >= 1e-30f)) return rsqrtf(fmaf(ss, p.inv_width, p.eps));
  double dd = 0.0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dd = fma((double)f[i][e], (double)f[i][e], dd);
  dd = row_sum(dd, wide, warps, bar);
  double root = sqrt(dd / (8.0 * p.vecs) + (double)p.eps);
  if (kNoEps && root > 0.0 && root < 0x1p-100) {
    root *= 0x1p64;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] *= 0x1p64f;
      const int v = threadIdx.x + i * (int)blockDim.x;
      if (stage && v < p.vecs) stage[v] = narrow8(f[i]);   // (exact)
    }
    if (stage) fence_async_shared();   // (the next row's copy lands there)
  }
  return (float)(1.0 / root);
}

// kVecs: vectors per thread.  The row's threads take vectors t, t + threads,
// ..; those past the row hold zeros.
template <int kVecs, bool kWide, bool kNoEps>
__global__ void __launch_bounds__(norm_max_threads(kVecs)) norm_kernel(const NormParams p) {
  __shared__ float s_part[2][32];
  __shared__ double s_wide[2][32];
  griddep_wait();
  griddep_launch_dependents();
  const int tpr = p.threads_per_row, warps = tpr >> 5;
  const int sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + sub;
  if (row >= p.rows) return;   // (whole groups)
  const int bar = 1 + sub, slot = sub * warps;
  bool on[kVecs];
  int at[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    at[i] = (t + i * tpr) * 8;
    on[i] = t + i * tpr < p.vecs;
  }
  // everything that the row needs is on its way before the first sum
  float x[kVecs][8], u[kVecs][8];
  uint4 g[kVecs], wp[kVecs], wz[kVecs];
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    uint4 yv = zero;
    if (p.y && on[i]) yv = *reinterpret_cast<const uint4*>(p.y + row * p.y_stride + at[i]);
    if (kWide) {
      float4 a = make_float4(0, 0, 0, 0), b = a;
      if (p.x && on[i]) {
        const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + row * p.x_stride + at[i]);
        a = src[0];
        b = src[1];
      }
      x[i][0] = a.x, x[i][1] = a.y, x[i][2] = a.z, x[i][3] = a.w;
      x[i][4] = b.x, x[i][5] = b.y, x[i][6] = b.z, x[i][7] = b.w;
    } else {
      uint4 xv = zero;
      if (p.x && on[i])
        xv = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + row * p.x_stride + at[i]);
      widen8(xv, x[i]);
    }
    widen8(yv, u[i]);
    g[i] = p.gate && on[i] ? *reinterpret_cast<const uint4*>(p.gate + row * p.gate_stride + at[i]) : zero;
    wp[i] = p.w_post && on[i] ? *reinterpret_cast<const uint4*>(p.w_post + at[i]) : zero;
    wz[i] = p.w_pre && on[i] ? *reinterpret_cast<const uint4*>(p.w_pre + at[i]) : zero;
  }
  if (p.w_post) {
    const float r = row_scale<kVecs, kNoEps>(u, s_part[0] + slot, s_wide[0] + slot, warps, bar, p);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float w[8];
      widen8(wp[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[i][e] = u[i][e] * r * (p.offset + w[e]);
    }
  }
  if (p.gate) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float w[8];
      widen8(g[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[i][e] *= w[e];
    }
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = p.x ? p.residual_scale * x[i][e] : 0.f;
      x[i][e] = p.y ? fmaf(p.branch_scale, u[i][e], a) : a;
    }
  if (p.x_out) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if (!on[i]) continue;
      if (kWide) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.x_out) + row * p.x_out_stride + at[i]);
        dst[0] = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
        dst[1] = make_float4(x[i][4], x[i][5], x[i][6], x[i][7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.x_out) + row * p.x_out_stride + at[i]) = narrow8(x[i]);
      }
    }
  }
  if (p.z) {
    const float r = row_scale<kVecs, kNoEps>(x, s_part[1] + slot, s_wide[1] + slot, warps, bar, p);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if (!on[i]) continue;
      float w[8], o[8];
      widen8(wz[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = x[i][e] * r * (p.w_pre ? p.offset + w[e] : 1.f);
      *reinterpret_cast<uint4*>(p.z + row * p.z_stride + at[i]) = narrow8(o);
    }
  }
}

// ---------------------------------------------------------------- many rows
// The same for many rows of a bf16 stream: CTAs of 512 threads' worth to an SM walk the rows, each
// with a ring of rows in shared memory that bulk copies fill rows ahead, and the
// weights in registers, so that the loads do not wait for a row's two sums.  A
// stage goes back when the row's stream stands in registers.
constexpr int kNsVecs = 4;                    // vectors of a thread
constexpr int kNsThreads = 256;               // of a CTA (at most)
constexpr int kNsMaxStages = 6;
constexpr int kNsSmem = 216 * 1024;           // of an SM's CTAs' rings

struct NsCfg {
  int32_t stages, stage_bytes, x_at, gate_at;   // a stage: y | x | gate (where each row has its own)
};

template <bool kNoEps>
__global__ void __launch_bounds__(kNsThreads, 2) norm_rows_kernel(const NormParams p, const NsCfg cfg) {
  constexpr int kVecs = kNsVecs;
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ float s_part[2][2][32];
  __shared__ double s_wide[2][2][32];
  __shared__ uint64_t s_full[kNsMaxStages];
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x, warps = blockDim.x >> 5;
  const int64_t step = gridDim.x;
  const int n = (int)((p.rows - (int64_t)blockIdx.x + step - 1) / step);   // rows of this CTA
  const bool own_gates = p.gate && p.gate_stride != 0;
  const uint32_t size = (uint32_t)p.vecs * 16u;
  const uint32_t bytes = (p.y ? size : 0u) + (p.x ? size : 0u) + (own_gates ? size : 0u);
  auto fetch = [&](int i) {   // (one thread)
    const int64_t row = blockIdx.x + i * step;
    uint8_t* st = s_ring + (i % cfg.stages) * cfg.stage_bytes;
    uint64_t* bar = &s_full[i % cfg.stages];
    mbar_arrive_expect_tx(bar, bytes);
    if (p.y) bulk_load(st, p.y + row * p.y_stride, size, bar);
    if (p.x) bulk_load(st + cfg.x_at, static_cast<const uint16_t*>(p.x) + row * p.x_stride, size, bar);
    if (own_gates) bulk_load(st + cfg.gate_at, p.gate + row * p.gate_stride, size, bar);
  };
  if (t == 0) {
    for (int s = 0; s < cfg.stages; ++s) mbar_init(&s_full[s], 1);
    s_abort = 0;
    fence_mbar_init();
    fence_proxy_async_global();
    for (int i = 0; i < cfg.stages && i < n; ++i) fetch(i);
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 wp[kVecs], wz[kVecs], g0[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = t + i * (int)blockDim.x;
    const bool on = v < p.vecs;
    wp[i] = p.w_post && on ? *reinterpret_cast<const uint4*>(p.w_post + v * 8) : zero;
    wz[i] = p.w_pre && on ? *reinterpret_cast<const uint4*>(p.w_pre + v * 8) : zero;
    g0[i] = p.gate && !own_gates && on ? *reinterpret_cast<const uint4*>(p.gate + v * 8) : zero;
  }
  __syncthreads();
  int k = 0;
  for (; k < n; ++k) {
    const int64_t row = blockIdx.x + k * step;
    uint8_t* st = s_ring + (k % cfg.stages) * cfg.stage_bytes;
    const int turn = k & 1;   // (sums of neighbouring rows stand apart: a barrier lies between a place's uses)
    bool ok = mbar_wait(&s_full[k % cfg.stages], (k / cfg.stages) & 1, abort_flag);
    float x[kVecs][8];
    float r = 1.f;
    if (p.w_post) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const int v = t + i * (int)blockDim.x;
        widen8(v < p.vecs ? reinterpret_cast<const uint4*>(st)[v] : zero, x[i]);
      }
      r = row_scale<kVecs, kNoEps>(x, s_part[turn][0], s_wide[turn][0], warps, 1, p, reinterpret_cast<uint4*>(st));
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int v = t + i * (int)blockDim.x;
      const bool on = v < p.vecs;
      float u[8], w[8];
      widen8(p.y && on ? reinterpret_cast<const uint4*>(st)[v] : zero, u);
      if (p.w_post) {
        widen8(wp[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = u[e] * r * (p.offset + w[e]);
      }
      if (p.gate) {
        widen8(own_gates ? (on ? reinterpret_cast<const uint4*>(st + cfg.gate_at)[v] : zero) : g0[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] *= w[e];
      }
      widen8(p.x && on ? reinterpret_cast<const uint4*>(st + cfg.x_at)[v] : zero, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = p.x ? p.residual_scale * w[e] : 0.f;
        x[i][e] = p.y ? fmaf(p.branch_scale, u[e], a) : a;
      }
    }
    // the stage is read: the next row that stands there may come
    if (!__syncthreads_and(ok)) break;
    if (t == 0 && k + cfg.stages < n) fetch(k + cfg.stages);
    if (p.x_out) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const int v = t + i * (int)blockDim.x;
        if (v >= p.vecs) continue;
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.x_out) + row * p.x_out_stride)[v] = narrow8(x[i]);
      }
    }
    if (p.z) {
      r = row_scale<kVecs, kNoEps>(x, s_part[turn][1], s_wide[turn][1], warps, 1, p);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const int v = t + i * (int)blockDim.x;
        if (v >= p.vecs) continue;
        float w[8], o[8];
        widen8(wz[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = x[i][e] * r * (p.w_pre ? p.offset + w[e] : 1.f);
        reinterpret_cast<uint4*>(p.z + row * p.z_stride)[v] = narrow8(o);
      }
    }
  }
  if (t == 0 && *abort_flag) {
    // what was issued lands before the CTA leaves (fewer copies than rows: the walk ended at row k)
    const RowRing ring(cfg.stages, n, k);
    for (int s = 0; s < ring.used(); ++s) drain_wait(&s_full[s], ring.last_parity(s), abort_flag);
    report_error(p.dev_error, HB_DEVERR_TIMEOUT);
  }
}

cudaError_t launch_rows(const NormParams& p, const NsCfg& cfg, int grid, int block, cudaStream_t st) {
  const auto kernel = p.eps > 0.f ? norm_rows_kernel<false> : norm_rows_kernel<true>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsSmem / 2);
  if (e != cudaSuccess) return e;
  return launch_serialized(kernel, (unsigned)grid, (unsigned)block, (size_t)cfg.stages * cfg.stage_bytes, st, p, cfg);
}

template <int kVecs>
cudaError_t launch(const NormParams& p, bool wide, unsigned grid, unsigned block, cudaStream_t st) {
  const auto kernel = p.eps > 0.f ? (wide ? norm_kernel<kVecs, true, false> : norm_kernel<kVecs, false, false>)
                                  : (wide ? norm_kernel<kVecs, true, true> : norm_kernel<kVecs, false, true>);
  return launch_serialized(kernel, grid, block, 0, st, p);
}

}  // namespace
}  // namespace hb

using namespace hb;

extern "C" hb_status hb_norm(const hb_norm_args* a, void* stream) {
  try {
    if (!a) return internal_fail(HB_ERR_INVALID_ARG, "args is NULL");
    if (a->reserved != 0) return internal_fail(HB_ERR_INVALID_ARG, "hb_norm_args.reserved must be 0");
    if (a->stream_type != HB_STREAM_BF16 && a->stream_type != HB_STREAM_FP32)
      return internal_failf(HB_ERR_INVALID_ARG, "unknown stream_type %d", a->stream_type);
    if (a->rows < 0 || a->width <= 0) return internal_failf(HB_ERR_SHAPE, "rows %d, width %d", a->rows, a->width);
    if (a->width % 8) return internal_failf(HB_ERR_UNSUPPORTED, "width %d: a multiple of 8 is needed", a->width);
    if (a->width > kNormMaxWidth)
      return internal_failf(HB_ERR_UNSUPPORTED, "width %d: at most %d", a->width, kNormMaxWidth);
    if (!a->x && !a->y) return internal_fail(HB_ERR_INVALID_ARG, "neither x nor y is given");
    if (!a->x_out && !a->z) return internal_fail(HB_ERR_INVALID_ARG, "neither x_out nor z is given");
    if (!a->y && (a->w_post || a->gate)) return internal_fail(HB_ERR_INVALID_ARG, "w_post and gate need y");
    if (!a->z && a->w_pre) return internal_fail(HB_ERR_INVALID_ARG, "w_pre needs z");
    if (!(a->eps >= 0.f && a->eps <= FLT_MAX)) return internal_failf(HB_ERR_INVALID_ARG, "eps %g", a->eps);
    if (!std::isfinite(a->residual_scale) || !std::isfinite(a->branch_scale) || !std::isfinite(a->weight_offset))
      return internal_fail(HB_ERR_INVALID_ARG, "scales and weight_offset must be finite");
    const int64_t n = a->rows, wide = a->stream_type == HB_STREAM_FP32 ? 4 : 2, w = a->width;
    const Operand x{a->x, n, w * wide, a->x_stride * wide, "x"}, y{a->y, n, w * 2, a->y_stride * 2, "y"},
        gate{a->gate, a->gate_stride ? n : 1, w * 2, a->gate_stride * 2, "gate"},
        w_post{a->w_post, 1, w * 2, 0, "w_post"}, w_pre{a->w_pre, 1, w * 2, 0, "w_pre"},
        x_out{a->x_out, n, w * wide, a->x_out_stride * wide, "x_out"}, z{a->z, n, w * 2, a->z_stride * 2, "z"};
    hb_status s;
    for (const Operand* o : {&x, &y, &gate, &w_post, &w_pre, &x_out, &z}) {
      if (o->p && (s = check_rows(*o)) != HB_OK) return s;
    }
    for (const Operand* out : {&x_out, &z})
      for (const Operand* in : {&x, &y, &gate, &w_post, &w_pre})
        if ((s = check_apart(*out, *in, in == &x || in == &y || (in == &gate && a->gate_stride))) != HB_OK) return s;
    if ((s = check_apart(x_out, z, false)) != HB_OK) return s;
    if (n == 0) return internal_ok();
    NormParams p{};
    int num_sms = 0;
    if ((s = internal_device(&p.dev_error, &num_sms)) != HB_OK) return s;
    p.rows = a->rows;
    p.vecs = a->width / 8;
    p.x = a->x;
    p.y = static_cast<const uint16_t*>(a->y);
    p.gate = static_cast<const uint16_t*>(a->gate);
    p.w_post = static_cast<const uint16_t*>(a->w_post);
    p.w_pre = static_cast<const uint16_t*>(a->w_pre);
    p.x_out = a->x_out;
    p.z = static_cast<uint16_t*>(a->z);
    p.x_stride = a->x_stride;
    p.y_stride = a->y_stride;
    p.gate_stride = a->gate_stride;
    p.x_out_stride = a->x_out_stride;
    p.z_stride = a->z_stride;
    p.eps = a->eps;
    p.residual_scale = a->residual_scale;
    p.branch_scale = a->branch_scale;
    p.offset = a->weight_offset;
    p.inv_width = 1.f / (float)a->width;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool fp32 = a->stream_type == HB_STREAM_FP32;
    auto launched = [&](cudaError_t e) {
      if (e != cudaSuccess) return internal_failf(HB_ERR_CUDA, "norm launch: %s", cudaGetErrorString(e));
      internal_note_other_launch(stream);
      internal_count_launch();
      return internal_ok();
    };
    NsCfg cfg{};
    cfg.x_at = p.y ? p.vecs * 16 : 0;
    cfg.gate_at = cfg.x_at + (p.x ? p.vecs * 16 : 0);
    cfg.stage_bytes = cfg.gate_at + (p.gate && p.gate_stride ? p.vecs * 16 : 0);
    // many rows: each CTA walks some of them, copies running ahead
    const int rows_block = ((p.vecs + kNsVecs - 1) / kNsVecs + 31) / 32 * 32;
    const int rows_ctas = std::min(16, 2 * kNsThreads / rows_block);
    cfg.stages = rows_block <= kNsThreads ? std::min(kNsMaxStages, (kNsSmem / rows_ctas - 2560) / cfg.stage_bytes) : 0;
    // measured, bf16 sum and norm: 9600 rows of 2048 29.0 us (a row per CTA 38.2), 2400 of 4096 15.9 (17.9), 2400 of
    // 8192 28.8 (32.1), 8191 gated ones of 4096 59.6 (62.8); but 2400 of 1024 6.4 (5.7), 512 of 4096 5.7 (5.1); fp32
    // streams, whose rows fill the rings: 2048 of 7168 39.3 (37.9)
    if (cfg.stages >= 2 && !fp32 && p.vecs >= 128 && n * a->width >= (4 << 20))
      return launched(launch_rows(p, cfg, (int)std::min<int64_t>(n, rows_ctas * num_sms), rows_block, st));
    // a vector per thread where the rows are few (the shortest chain); two or
    // four where they are many or wide
    int per = 1;
    while (per < 4 && (p.vecs > norm_max_threads(per) * per || (n > 2 * num_sms && p.vecs > 128 * per))) per *= 2;
    p.threads_per_row = ((p.vecs + per - 1) / per + 31) / 32 * 32;
    const int rows_per_cta = std::max(1, std::min(8, (n > 2 * num_sms ? 256 : 32) / p.threads_per_row));
    const unsigned grid = (unsigned)((n + rows_per_cta - 1) / rows_per_cta);
    const unsigned block = (unsigned)(rows_per_cta * p.threads_per_row);
    return launched(per == 1   ? launch<1>(p, fp32, grid, block, st)
                    : per == 2 ? launch<2>(p, fp32, grid, block, st)
                               : launch<4>(p, fp32, grid, block, st));
  } catch (...) {
    return internal_fail(HB_ERR_CUDA, "unexpected exception in hb_norm");
  }
}
