// E4M3 codes of bf16 values (the rule is stated in fp8_quant.hip).  Included by
// HIP sources only.
#pragma once
#include "common.h"

namespace moe {

constexpr float kE4M3Max = 448.0f;

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Two fp32 values -> two E4M3 codes in the low 16 bits (first value low).
__device__ __forceinline__ uint32_t fp8x2(float a, float b) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu;
}

__device__ __forceinline__ float quant_input(float v, float s) {
  return fminf(fmaxf(v / s, -kE4M3Max), kE4M3Max);
}

// Eight bf16 (one 16-byte word) -> their eight E4M3 codes under scale s.
__device__ __forceinline__ uint2 quant8(uint4 v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = fp8x2(quant_input(bf16_to_f32(w[i] & 0xFFFFu), s), quant_input(bf16_to_f32(w[i] >> 16), s));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// |v| of the eight bf16 in v, widened to fp32 bits, maximum of them (the order
// of non-negative floats is the order of their bits).
__device__ __forceinline__ uint32_t abs_max8(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(w[i] << 17 >> 1, w[i] & 0x7FFF0000u));
  return m;
}

}  // namespace moe
