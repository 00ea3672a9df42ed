// e4m3 values with power-of-two block scales: the scale's exponent and the conversion, shared by
// the quantizer and the gate/up product's epilogue.
#pragma once

#include "common.h"

namespace moe {

constexpr int kScaleF32 = 0, kScaleE8M0 = 1;  // moe_scale_type
constexpr int kScaleBlock = 128;

// Magnitudes are compared as the bits of |x| (sign cleared): an order that puts infinity above
// every number and NaN above infinity, so no special value is lost in a maximum.
__device__ inline uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;

// The least e >= -126 with amax <= 448 * 2^e (448 = 1.75 * 2^8), 0 for amax = 0.  amax finite.
__device__ inline int scale_exponent(uint32_t amax) {
  const int e = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return amax == 0 ? 0 : max(e, -126);
}

// A block's scale in its storage type at scale[i]; non-finite blocks get NaN.
__device__ inline void store_scale(void* scale, int64_t i, int scale_type, int e, bool finite) {
  if (scale_type == kScaleE8M0)
    static_cast<uint8_t*>(scale)[i] = finite ? (uint8_t)(e + 127) : (uint8_t)255;
  else
    static_cast<float*>(scale)[i] =
        __uint_as_float(finite ? (uint32_t)(e + 127) << 23 : 0x7fc00000u);
}

// 2^-e for -126 <= e <= 126.
__device__ inline float inv_scale(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

// Four floats of magnitude at most 448 to four e4m3 bytes, rounded to nearest even (the
// instruction's rounding).
__device__ inline uint32_t pack_e4m3(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
constexpr uint32_t kNan4 = 0x7f7f7f7fu;  // four e4m3 NaN

}  // namespace moe
