// mx8_quant.cuh -- 8-bit quantisation with power-of-two scales (device functions).
//
// A group of values (32 of a row for the RMS norm's output; one head's vector of
// one token for the key-value cache) is held as E4M3 codes (4 exponent and 3
// mantissa bits, largest value 448, no infinity, 0x7F is NaN) and one E8M0 byte
// b (value 2^(b-127), 255 is NaN).  The scale is X = 2^e with the smallest e such
// that max|v| <= 448 X, clamped to -127 .. 127 (an all-zero group has e = -127), and
// a code is v / X rounded to nearest even.  Nothing saturates, unlike under the
// rule floor(log2 max|v|) - 8, which cuts the top eighth of a binade off; a
// power of two costs E4M3 no precision, since its spacing is relative, and it
// leaves code * X exact in bf16 (above 2^-124).  A group holding a NaN or an
// infinity has the byte 255 and codes 0x7F: it reads back as NaN throughout.
#pragma once
#include <stdint.h>

#include "mx_quant.cuh"

namespace k3moe {

constexpr uint32_t kMx8Bad = 255u;  // E8M0 NaN

// E8M0 byte of a group from its largest magnitude, given as the largest of its
// values' bit patterns with the sign removed (so a NaN or an infinity is seen).
__device__ __forceinline__ uint32_t mx8_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return kMx8Bad;
  // floor(log2 amax) + 127, 0 for subnormal values; 448 = 1.75 * 2^8
  const int ex = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u);
  return static_cast<uint32_t>(max(0, min(254, ex)));
}

// 1 / X for a scale byte below 255.
__device__ __forceinline__ float mx8_inv_scale(uint32_t byte) { return mx_pow2(127 - static_cast<int>(byte)); }

// Two values rounded to bf16 (to nearest even), `lo` in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two values (already divided by X) -> two codes, `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight values -> eight codes of a group with scale byte `byte` (0x7F codes for 255).
__device__ __forceinline__ uint2 mx8_codes(const float (&v)[8], uint32_t byte) {
  if (byte == kMx8Bad) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float r = mx8_inv_scale(byte);
  return make_uint2(e4m3x2(v[0] * r, v[1] * r) | (e4m3x2(v[2] * r, v[3] * r) << 16),
                    e4m3x2(v[4] * r, v[5] * r) | (e4m3x2(v[6] * r, v[7] * r) << 16));
}

// Four codes -> two f16x2 registers (exact), code 0 in the low half of the first.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t &a, uint32_t &b) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(w));
}

}  // namespace k3moe
