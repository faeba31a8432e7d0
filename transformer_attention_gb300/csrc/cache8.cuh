// The 8-bit KV cache's numbers: e4m3 values in blocks of kC8Block slots, one
// fp32 scale per block, kv head and K' or V.  A stored byte n in a block of
// scale s stands for e4m3(n) * s.
//
// Why e4m3 with a power-of-two scale: e4m3 rounds relative to the value, so
// the scale only has to bring a block's largest number under 448; any finer
// choice of it moves no rounding.  With a power of two, a block whose scale
// grows by 2^k (a later token larger than the block's first ones) keeps every
// number that stays normal exactly, and every value is an exact fp32 product.
// With exponents from -15 up a value is a multiple of 2^-24, fp16's last
// step, so reading a cache back as fp16 rounds nothing below fp16's largest.
//
// The kernels over this cache read what another launch may have written
// (numbers, scales, weights, scratch, positions and padding of the slots and
// of the queries) past L1, by __ldcg: a kernel starts while the one before it
// runs (pdl_enter), so that a line which that one still reads into an SM's L1
// may not be dropped again before this one.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace g3 {

constexpr int kC8Block = 64;
constexpr float kC8MinScale = 3.0517578125e-05f;   // 2^-15

// Smallest 2^e >= 2^-15 with amax <= 448 * 2^e (448 = 1.75 * 2^8), for a
// finite amax >= 0.
__device__ __forceinline__ float c8_scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -15 ? -15 : e;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The two e4m3 numbers of the low 16 bits as fp16 (exact; NaN stays NaN).
__device__ __forceinline__ uint32_t c8_half2(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(h)
      : "r"(two));
  return h;
}
__device__ __forceinline__ uint32_t c8_half2_hi(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}"
      : "=r"(h)
      : "r"(two));
  return h;
}
__device__ __forceinline__ float2 c8_float2(uint32_t two) {
  const uint32_t h = c8_half2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four fp32 values to four e4m3 bytes, to nearest even; beyond 448 (only an
// infinite input, given the scale) to 448, NaN to NaN.
__device__ __forceinline__ uint32_t c8_pack4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Four e4m3 bytes times `ratio`, rounded to e4m3 again.
__device__ __forceinline__ uint32_t c8_rescale4(uint32_t n, float ratio) {
  const float2 lo = c8_float2(n), hi = c8_float2(n >> 16);
  return c8_pack4(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
}

}  // namespace g3
