// kv8.cuh -- the 8-bit KV cache: e4m3 values with one exponent per (page, kv
// head), shared by the append and the attention over it.
//
// A page's element of kv head h stands for  value * 2^exp[page][h],  value an
// e4m3 number (4 significant bits, largest 448, smallest step 2^-9).  The
// scale is a power of two on purpose.  e4m3 is itself a floating-point
// format, so a finer scale would gain nothing but the last fraction of a bit
// of range; a power of two makes value * scale exact in bf16 and fp16-and-
// exponent alike, and a page whose scale has to grow keeps its values but for
// those that fall below the smallest normal number.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hb_internal.h"
#include "ptx.cuh"

namespace hb {

// Exponents in use.  448 * 2^64 = 8e21 is far above any key or value; past
// it a value is held at the largest one.  Inside this range the scales and
// the sums of the attention stay clear of fp32's ends.
constexpr int kKv8MinExp = -64, kKv8MaxExp = 64;

__device__ __forceinline__ int kv8_exp(int8_t e) {
  return min(max((int)e, kKv8MinExp), kKv8MaxExp);
}

// 2^e for -126 <= e <= 127; 0 below.
__device__ __forceinline__ float pow2i(int e) {
  return __uint_as_float((uint32_t)max(0, e + 127) << 23);
}

// The smallest e with amax <= 448 * 2^e, for amax given as the bits of a
// finite non-negative bf16: amax = (1 + M / 128) 2^(E - 127), 448 = 1.75 * 2^8.
__device__ __forceinline__ int kv8_need_exp(uint32_t bf16_bits) {
  const int E = (int)(bf16_bits >> 7), M = (int)(bf16_bits & 127u);
  return min(max(E - 135 + (M > 96 ? 1 : 0), kKv8MinExp), kKv8MaxExp);   // zero: the smallest
}

// Two fp32 to e4m3 (round to nearest even, held at +-448, NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 (the low 16 bits of v) to fp16, exactly.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return r;
}
__device__ __forceinline__ float2 f32x2_of_f16x2(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Two fp32 to fp16 (round to nearest even).
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// c[16x8] += a[16x16] * b[16x8], fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// *p += v at device scope, as a release of everything ordered before it and
// an acquire of what the others released there.
__device__ __forceinline__ int atom_add_acq_rel(int32_t* p, int v) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// A byte through L2 (another kernel may have written it since this SM's L1
// last saw its line).
__device__ __forceinline__ int8_t ldcg_s8(const int8_t* p) {
  int32_t v;
  asm volatile("ld.global.cg.s8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return (int8_t)v;
}

}  // namespace hb
