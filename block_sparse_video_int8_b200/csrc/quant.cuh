// quant.cuh -- the step from a scaled value to its INT8 code, shared by the per-block quantisers
// (quant_pool.cu) and the per-token quantiser of the paged cache (paged_kv.cu).
#pragma once

#include "common.cuh"

namespace bsva {

constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: q + kMagic rounds q to an integer, half to even
// Half-integer guard band. With rcp = fl(1/s) and q = fl(x * rcp), |x/s| <= 127 + 2^-16 gives
// |q - x/s| <= 127.0001 * (2^-23 + 2^-48) < 1.52e-5, and the IEEE quotient fl(x/s) lies within
// 2^-18 < 3.9e-6 of x/s, so q and fl(x/s) round to the same integer unless q is within 1.9e-5 of
// a half-integer (ties of fl(x/s) included). Chunks with such an element take the exact division.
constexpr float kBand = 0.5f - 4e-5f;

// |a| max of two bf16x2 words (sign bits of the result are meaningless and masked later).
__device__ __forceinline__ uint32_t bmax_abs(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float bmax_fold(uint32_t m) {
  return fmaxf(__uint_as_float((m & 0x7FFFu) << 16), __uint_as_float(m & 0x7FFF0000u));
}

// Exact step for one element: code n of rint_half_even(fl32(x / s)), returned as the float
// kMagic + n (the bit pattern the fast path produces; its low byte is n as int8).
__device__ __forceinline__ float quant_exact(float x, float s) {
  const int n = (s == 0.f) ? 0 : __float2int_rn(__fdiv_rn(x, s));
  return __int_as_float(0x4B400000 + n);
}

}  // namespace bsva
