// Values that trade places between the lanes of a wave, so that stores go out in
// whole lines.  Included by HIP sources only.
#pragma once
#include "common.h"

namespace moe {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2_t v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// The upper 32 lanes' a change places with the lower lanes' b; the odd rows'
// (of 16 lanes) a with the even rows' b; within every 16 lanes, the upper
// eight's a with the lower eight's b.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap_rows16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap_rows8(uint32_t& a, uint32_t& b) {
  constexpr int kRor8 = 0x128;  // row_ror:8; the bank masks write one half of the 16
  const uint32_t a0 = a;
  a = (uint32_t)__builtin_amdgcn_update_dpp((int)a, (int)b, kRor8, 0xF, 0xC, false);
  b = (uint32_t)__builtin_amdgcn_update_dpp((int)b, (int)a0, kRor8, 0xF, 0x3, false);
}

// Where a lane's 16 bytes lie in a group of eight rows x 64 columns.
__device__ __forceinline__ int line_row(int lane) { return lane & 7; }
__device__ __forceinline__ int line_col(int lane) {
  return 32 * ((lane >> 3) & 1) + 16 * ((lane >> 4) & 1) + 8 * (lane >> 5);
}

}  // namespace moe
