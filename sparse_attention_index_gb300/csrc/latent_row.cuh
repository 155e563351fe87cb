// e4m3 codes of a latent cache row widened to bf16, exactly: its scales are powers of two.
#pragma once

#include "dsa_common.cuh"

namespace dsa {

// 2^7 as bf16: the largest scale that widens in one step
constexpr uint32_t kScaleMost = 134u << 7;

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Four e4m3 bytes to bf16. The 7 magnitude bits, moved to the top of the bf16 mantissa and the
// bottom of its exponent, are the value times 2^-120 (biases 127 and 7; the subnormals of one are
// subnormals of the other), so one exact multiply by 2^(120 + k), twice in `up`, widens and scales.
// The bytes come out as (0, 2) and (1, 3), which needs no byte permutation.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t up, uint32_t& even, uint32_t& odd) {
  even = mul_bf16x2(((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u), up);
  odd = mul_bf16x2(((w >> 4) & 0x07f007f0u) | (w & 0x80008000u), up);
}

// The same with the bytes in order, two at a time: each byte under its own sign, which prmt spreads out,
// moved up by four bits.
__device__ __forceinline__ void widen4_in_order(uint32_t w, uint32_t up, uint32_t& lo, uint32_t& hi) {
  uint32_t a, b;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(a) : "r"(w));
  asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(b) : "r"(w));
  lo = mul_bf16x2((a << 4) & 0x87f087f0u, up);
  hi = mul_bf16x2((b << 4) & 0x87f087f0u, up);
}

// `up` of a scale given as bf16 bits (at most kScaleMost)
__device__ __forceinline__ uint32_t widen_factor(uint32_t scale) {
  return (min(scale, kScaleMost) + (120u << 7)) * 0x10001u;
}
// what is left to multiply by for a scale above kScaleMost: 2^(k - 7), or NaN
__device__ __forceinline__ uint32_t widen_rest(uint32_t scale) {
  return scale > 0x7f80u ? 0x7fff7fffu : (scale - (7u << 7)) * 0x10001u;
}

}  // namespace dsa
