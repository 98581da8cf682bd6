// Microscaled 4-bit floats on the device, shared by the exchange kernels and
// the product: blocks of 32 consecutive values of a row, 16 bytes of codes (two
// a byte, the first in the low half) and one scale byte s, the power of two
// 2^(s - 127), 255 a NaN.  A code is a sign, two bits of exponent and one of
// mantissa: 0, 1/2, 1, 3/2, 2, 3, 4, 6.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bf16.h"

namespace sbp {

constexpr int kMx4Block = 32;

inline int64_t mx4_blocks(int64_t cols) { return (cols + kMx4Block - 1) / kMx4Block; }

// The scale as the conversion instructions take it: a binary32 with exponent
// field s (0 stands for 2^-127, 255 for NaN).
__device__ __forceinline__ float mx4_scale(uint32_t s) { return __uint_as_float(s << 23); }

// Two codes (byte B of w) as values; exact in both types.
template <int B>
__device__ __forceinline__ void mx4_pair(uint32_t w, float scale, float& a, float& b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, B);
  a = v.x;
  b = v.y;
}
template <int B>
__device__ __forceinline__ uint32_t mx4_pair_bf16(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, B));
}
__device__ __forceinline__ void mx4_octet(uint32_t w, float scale, float (&v)[8]) {
  mx4_pair<0>(w, scale, v[0], v[1]);
  mx4_pair<1>(w, scale, v[2], v[3]);
  mx4_pair<2>(w, scale, v[4], v[5]);
  mx4_pair<3>(w, scale, v[6], v[7]);
}

}  // namespace sbp
