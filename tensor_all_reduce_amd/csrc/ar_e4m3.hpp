// E4M3 (OCP "FN") scale arithmetic shared by the quantising kernels.
#pragma once

#include "ar_device.hpp"

namespace ar {

// Largest of the 4 values held by one quad of lanes (lanes 4q..4q+3).
// DPP quad permutations [1,0,3,2] and [2,3,0,1]; every lane must be active.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  return v;
}

// Scale exponent k from the binary32 bits A of the block's largest finite
// magnitude: the smallest k in [-127, 127] with A <= 448 * 2^k.  For a
// normal A = (1 + F/2^23) * 2^(E-127) and 448 = 1.75 * 2^8, that is E - 135,
// plus one when the significand exceeds 1.75 (F > 0x600000).  Zero and
// binary32 subnormals (below 2^-126, far below 448 * 2^-127) give -127;
// the largest finite bf16 gives 120, so no upper clamp is reached.
__device__ __forceinline__ int fp8_scale_exp(uint32_t A) {
  const int E = (int)(A >> 23);
  if (E == 0) return -127;
  const int k = E - 135 + ((A & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return k < -127 ? -127 : k;
}

// Largest of the 16 values held by one row of lanes (lanes 16q..16q+15):
// the quad maximum, then DPP half-row and row mirrors.  Every lane must be
// active.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = quad_max(v);
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  return v;
}

// Scale of a block of 128 whose largest finite magnitude has the binary32
// bits A.  F32: s = max(amax / 448, 2^-126), one binary32 division, and the
// codes are those of x * (1 / s): the floor keeps s normal and 1 / s finite,
// and the reciprocal, formed once for 128 elements, replaces 128 divisions
// (x * (1 / s) is within 1.5 binary32 ulps of x / s, 2^-19 of the spacing of
// the codes).  E8M0: s = 2^k, k as fp8_scale_exp, and x * 2^-k is exact.
struct BlockScale {
  float inv;       // multiplies an element before its conversion
  uint32_t kept;   // the stored scale: binary32 bits, or the byte k + 127
};
template <bool E8M0>
__device__ __forceinline__ BlockScale block_scale(uint32_t A) {
  if constexpr (E8M0) {
    const int k = fp8_scale_exp(A);
    return BlockScale{__builtin_ldexpf(1.0f, -k), (uint32_t)(k + 127)};
  } else {
    const float s = fmaxf(__uint_as_float(A) / 448.0f, 0x1p-126f);
    return BlockScale{1.0f / s, __float_as_uint(s)};
  }
}

// Binary32 bits of |f| where f is finite, else 0: infinities and NaN take no
// part in a block's largest magnitude.
__device__ __forceinline__ uint32_t finite_mag(float f) {
  const uint32_t a = __float_as_uint(f) & 0x7FFFFFFFu;
  return a < 0x7F800000u ? a : 0u;
}

// Codes of 4 elements times inv, little-endian; 0x7F for a NaN or infinity.
// |f * inv| exceeds 448 by at most the roundings of s and 1 / s, which the
// conversion rounds back to 448.
__device__ __forceinline__ uint32_t codes4_scaled(const float* f, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0] * inv, f[1] * inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(f[2] * inv, f[3] * inv, w, true);
  uint32_t bad = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if ((__float_as_uint(f[j]) & 0x7FFFFFFFu) >= 0x7F800000u) bad |= 0xFFu << (8 * j);
  return ((uint32_t)w & ~bad) | (0x7F7F7F7Fu & bad);
}

}  // namespace ar
