// The 4-bit latent format: blocks of 16 features, sixteen E2M1 codes and one E4M3 scale,
//   value = code * scale * latent_scale,   latent_scale a power of two for the whole cache.
// Feature 2i of a row is the low half of byte i.  An E2M1 code has two significant bits and an E4M3
// scale four, so code * scale has at most six: it is exact in fp16 (range 2^-10 .. 2688), in bf16
// and in fp32, and reading a row back never rounds.
#pragma once

#include <stdint.h>

namespace mla {
namespace fp4 {

constexpr int kBlock = 16;  // features of one scale

// Eight codes (one word) to four fp16 pairs.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Eight codes (one word) to four bf16 pairs: the bytes of a magnitude are looked up by a byte
// permutation (its selectors are the codes), the sign bits come from its sign-replicating mode.
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t (&h)[4]) {
  const uint32_t mag = w & 0x77777777u, sgn = w & 0x88888888u;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t m = mag >> (16 * k), s = sgn >> (16 * k);
    // bf16 of 0 .5 1 1.5 2 3 4 6: 0000 3f00 3f80 3fc0 4000 4040 4080 40c0
    const uint32_t lo = __byte_perm(0xc0800000u, 0xc0804000u, m);
    const uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, m);
    uint32_t neg;  // 0x80 (plus) or 0xff (minus) in each byte
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(neg) : "r"(0x80u), "r"(s));
    const uint32_t top = hi | ((neg << 1) & 0x80808080u);
    h[2 * k] = __byte_perm(lo, top, 0x5140);
    h[2 * k + 1] = __byte_perm(lo, top, 0x7362);
  }
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two E4M3 scales (low and high byte) to an fp16 pair.
__device__ __forceinline__ uint32_t scales_to_f16(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}" : "=r"(h) : "r"(two));
  return h;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// (lo, hi) to two E2M1 codes in one byte / two E4M3 scales in one halfword: nearest, ties to even,
// saturating; a NaN scale stays NaN (0x7f).
__device__ __forceinline__ uint32_t to_codes(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t to_scales(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}

// The value of one E4M3 scale (0 .. 448, NaN for 0x7f); the sign bit is never set by the append.
__device__ __forceinline__ float scale_value(uint32_t s8) {
  const uint32_t h = scales_to_f16(s8 & 0xffu);
  float f;
  asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

}  // namespace fp4
}  // namespace mla
