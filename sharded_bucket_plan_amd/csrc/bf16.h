// bf16 <-> binary32 on the device, shared by the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sbp {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_one(uint16_t h) {
  return __uint_as_float(static_cast<uint32_t>(h) << 16);
}

// binary32 -> bf16 bits: nearest, ties to even; NaN kept (quiet bit set).
__device__ __forceinline__ uint32_t bf16_rne(float x) {
  const uint32_t u = __float_as_uint(x);
  const uint32_t rounded = (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
  const uint32_t quiet = (u >> 16) | 0x40u;
  return __builtin_isnan(x) ? quiet : rounded;  // a select, not a branch
}

}  // namespace sbp
