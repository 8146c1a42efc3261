// Conversions shared by the rotated append, the 4-bit gather and attention:
// e2m1 codes (4 bits: sign, two exponent bits, one mantissa bit; magnitudes
// 0, 0.5, 1, 1.5, 2, 3, 4, 6) with one e4m3fn scale per 16 dims, and the fp32 <->
// 16-bit roundings.
#pragma once

#include "kv_device.cuh"

namespace kvimpl {

constexpr int kFp4Block = KV_FP4_BLOCK;
constexpr float kSixth = 1.0f / 6.0f;  // fl(1/6): a block's largest magnitude maps to the code 6

// Eight fp32 values to eight e2m1 codes, value i in bits 4i .. 4i+3: nearest,
// ties to the even code, saturating at +-6; NaN becomes +6.
__device__ __forceinline__ uint32_t e2m1x8(const float* x) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Eight e2m1 codes (32 bits) to four f16x2 words, exact; word i holds dims 2i, 2i + 1.
__device__ __forceinline__ void f16x2_from_e2m1x8(uint32_t c, uint32_t* out) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(c));
}

// Two e4m3fn codes (low 16 bits) to an f16x2 word, exact.
__device__ __forceinline__ uint32_t f16x2_from_e4m3x2(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(c)));
  return r;
}

// One e4m3fn code to fp32, exact.
__device__ __forceinline__ float f32_from_e4m3(uint32_t c) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(f16x2_from_e4m3x2(c & 0xFFu))));
}

// Two fp32 values rounded to nearest-even bf16 / fp16 (lo in the low half); NaN
// becomes 0x7FFF, fp16 overflow an infinity.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, bool bf16) {
  uint32_t r;
  if (bf16) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  } else {
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  }
  return r;
}

__device__ __forceinline__ float2 unpack2(uint32_t w, bool bf16) {
  return bf16 ? widen2<true>(w) : widen2<false>(w);
}

__device__ __forceinline__ uint16_t round16(float x, bool bf16) {
  return static_cast<uint16_t>(pack2(x, 0.0f, bf16) & 0xFFFFu);
}

__device__ __forceinline__ float widen16(uint16_t h, bool bf16) {
  return bf16 ? __uint_as_float(static_cast<uint32_t>(h) << 16) : __half2float(__ushort_as_half(h));
}

// The e4m3fn block scale of a largest magnitude (>= 0), and the reciprocal of
// its value in fp32 (0 for a zero scale).
__device__ __forceinline__ uint32_t fp4_block_scale(float amax, float* recip) {
  const uint32_t c = e4m3x2(__fmul_rn(amax, kSixth), 0.0f) & 0xFFu;
  const float s = f32_from_e4m3(c);
  *recip = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
  return c;
}

}  // namespace kvimpl
