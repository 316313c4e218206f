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

}  // namespace hb
