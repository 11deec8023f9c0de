// gsg_mx.cuh -- the microscaled block rule shared by the weight packer, the activation quantizer and
// the norm.
//
// A block is 32 consecutive values along K with one power-of-two scale 2^e, stored as the byte e + 127
// (UE8M0), and 32 codes: E2M1 (largest value 6 = 1.5 * 2^2) or E4M3 (448 = 1.75 * 2^8).  With b the
// block's largest magnitude,
//     e = clamp(floor(log2 b) - emax, -127, 127),  emax = 2 (E2M1) or 8 (E4M3);  e = -127 for b = 0
//     code = RNE(v / 2^e), saturating at the largest value
// (the rule of the OCP microscaling formats).  floor(log2 b) is b's exponent field and v / 2^e a product
// with a power of two, so the whole rule is exact up to the one rounding to the code.
#pragma once

#include "gsg_internal.cuh"

namespace gsg {

// Scale byte of a block whose largest magnitude has these fp32 bits.  (A subnormal maximum has exponent
// field 0: its true exponent is lower still, and both clamp to -127.)
template <int kBits>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  constexpr int emax = kBits == 8 ? 8 : 2;
  return (uint32_t)max((int)(amax_bits >> 23) - emax, 0);
}
// 2^-e for the scale byte e + 127: e is in [-127, 125], so the exponent field 254 - byte is that of a
// normal number.
__device__ __forceinline__ float mx_inv_scale(uint32_t sc) { return __uint_as_float((254u - sc) << 23); }

// Four values -> four E4M3 codes, v[i] in byte i: round to nearest even, saturating at 448.
__device__ __forceinline__ uint32_t e4m3_encode4_cvt(float v0, float v1, float v2, float v3) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
  return r;
}

// Largest magnitude's bits (sign dropped) of a value, as an unsigned maximum: infinities and NaN stay
// the largest, so one test of the block's maximum finds them.
constexpr uint32_t kF32Inf = 0x7F800000u;
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace gsg
