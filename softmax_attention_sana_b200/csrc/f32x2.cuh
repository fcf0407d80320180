// Small device helpers of the windowed anchor and the query/key norm: base-2
// exponentials, packed fp32 pairs, maxima that keep NaN, shared-memory alignment.
#pragma once

#include "sana_common.cuh"

namespace sana {

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  const uint32_t a = smem_u32(p);
  return p + ((1024u - (a & 1023u)) & 1023u);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- packed fp32 (f32x2) helpers: one instruction for two lanes of math
__device__ __forceinline__ uint64_t pk2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void up2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Maxima that are NaN where an operand is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 2^x for two x <= 0 (or a little above) on the FMA pipe: n = round(x) in the low
// mantissa bits of x + 1.5 * 2^23, a cubic on [-1/2, 1/2] (7.5e-5 relative), times
// 2^n (so that NaN stays NaN).  Below -126 counts as -126: nothing in bf16 or beside 1.
__device__ __forceinline__ void exp2_pair(uint64_t x, float& y0, float& y1) {
  float a, b;
  up2(x, a, b);
  const uint64_t v = pk2(max_nan(a, -126.f), max_nan(b, -126.f)), c = pk2(12582912.f, 12582912.f);
  const uint64_t t = add2(v, c);
  const uint64_t f = sub2(v, sub2(t, c));
  uint64_t p = fma2(pk2(0.055170517f, 0.055170517f), f, pk2(0.24260856f, 0.24260856f));
  p = fma2(p, f, pk2(0.69326097f, 0.69326097f));
  p = fma2(p, f, pk2(0.99992824f, 0.99992824f));
  float t0, t1;
  up2(t, t0, t1);
  const float e0 = __uint_as_float(__float_as_uint(t0) * 8388608u + 0x3f800000u);  // 2^n
  const float e1 = __uint_as_float(__float_as_uint(t1) * 8388608u + 0x3f800000u);
  up2(mul2(p, pk2(e0, e1)), y0, y1);
}

}  // namespace sana
