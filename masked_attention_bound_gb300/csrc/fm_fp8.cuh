// What the kernels of the 8-bit cache share: e4m3 codes and their scales.
#pragma once
#include <cstdint>

#include "fm.h"
#include "fm_ptx.cuh"

namespace fm {

constexpr int kScaleBlock = FM_SCALE_BLOCK;        // tokens of a head that share a scale
constexpr int kScaleShift = 4;

// A scale as every kernel reads it: within [2^-60, 2^60] (NaN: 2^-60).  With
// that no product of scales overflows, log2 of one is finite, and a block
// whose scale was never written cannot put a NaN on what a row does not see.
constexpr float kLeastScale = 0x1p-60f, kMostScale = 0x1p60f;
__device__ __forceinline__ float clamp_scale(float s) { return fminf(fmaxf(s, kLeastScale), kMostScale); }

// The least power of two s with amax / s <= 448 = 1.75 * 2^8, within the
// range above: the exponent of amax less 8, and one more if its mantissa is
// past 1.75.  A power of two: requantising a block to a larger scale then
// rounds only what falls below the smallest normal code.
__device__ __forceinline__ float scale_for(float amax) {
  const int e = static_cast<int>((__float_as_uint(amax) + 0x1fffffu) >> 23) - 127 - 8;
  return __int_as_float((min(max(e, -60), 60) + 127) << 23);
}

// Two codes (low 16 bits) as two f16, exactly: f16 holds every e4m3 value.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ float2 float2_of_f16x2(uint32_t h) {
  float lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four codes times a factor, rounded to codes again.
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t c, float f) {
  const float2 a = float2_of_f16x2(f16x2_of_e4m3x2(c)), b = float2_of_f16x2(f16x2_of_e4m3x2(c >> 16));
  return pack_e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}
__device__ __forceinline__ uint4 rescale_e4m3x16(uint4 x, float f) {
  return make_uint4(rescale_e4m3x4(x.x, f), rescale_e4m3x4(x.y, f), rescale_e4m3x4(x.z, f),
                    rescale_e4m3x4(x.w, f));
}

// The bytes of x that are NaN (e4m3 has no infinities), as 0xff each.
__device__ __forceinline__ uint32_t e4m3x4_nan(uint32_t x) { return __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu); }

}  // namespace fm
