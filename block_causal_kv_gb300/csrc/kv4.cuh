// The 4-bit K/V cache: its page layout and the conversions between floats and codes.
//
// Sixteen consecutive elements of one token's head row share one e4m3 scale; an
// element is one e2m1 code (sign, two exponent bits, one mantissa bit: 0, 0.5, 1,
// 1.5, 2, 3, 4, 6). With y = x * 2^-e (e: the caller's exponent of the K or V pool),
//   scale = e4m3(max |y| / 6),  code = e2m1(y / scale),  value = code * scale * 2^e,
// each conversion to nearest, ties to even, saturating. A code has two significant
// bits and a scale four, so code * scale has at most six: exact in fp16 and bf16
// (which is why dequantised tiles feed fp16 matrix products without a rounding).
//
// One page of one KV head (B tokens, D dims; bytes):
//   K codes   [D / 32][B][16]  byte i of chunk c of token t: dims 32c + 2i (low nibble), +1
//   V codes   [D][B / 2]       byte i of dim d: tokens 2i (low nibble), 2i + 1
//   K scales  [B][D / 16]
//   V scales  [D / 16][B]
// The layout is the one the tensor-core attention wants: a thread that owns a token's
// K row reads 16-byte pieces whose neighbours in a warp are contiguous (no bank
// conflicts), and a thread that owns a V dim reads that dim's codes of the page as
// one word, already in the order of the transposed V tile. K and V of a page are one
// contiguous piece of B * D * 9/8 bytes, so a page is one bulk copy.
#pragma once

#include "d2f_internal.cuh"

namespace d2f {

struct Kv4Layout {
  int D, B;
  __host__ __device__ int page_bytes() const { return B * D + B * D / 8; }
  __host__ __device__ int v_codes() const { return B * D / 2; }
  __host__ __device__ int k_scales() const { return B * D; }
  __host__ __device__ int v_scales() const { return B * D + B * D / 16; }
};

#ifdef __CUDACC__
// The larger of two floats, NaN if either is.
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// e4m3 bits of x >= 0: nearest, ties to even, saturating at 448; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3_bits(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}

// Two e4m3 values (low byte first) as packed halves, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t bits16) {
  uint32_t r;
  const uint16_t b = (uint16_t)bits16;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(b));
  return r;
}

__device__ __forceinline__ float half_lo(uint32_t h2) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h2));
  return f;
}
__device__ __forceinline__ float half_hi(uint32_t h2) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(h2));
  return f;
}

// Two e2m1 codes (low nibble first) as packed halves, exact.
__device__ __forceinline__ uint32_t e2m1x2_to_half2(uint32_t bits8) {
  uint32_t r;
  asm("{\n\t.reg .b8 t, u0, u1, u2;\n\tmov.b32 {t, u0, u1, u2}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
      : "=r"(r)
      : "r"(bits8));
  return r;
}

// Codes of (lo, hi) in one byte, low nibble first: nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t e2m1x2_bits(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// The same of eight halves (four pairs), as one word.
__device__ __forceinline__ uint32_t half8_to_codes(const uint32_t (&h)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 a, %1;\n\tcvt.rn.satfinite.e2m1x2.f16x2 b, %2;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 c, %3;\n\tcvt.rn.satfinite.e2m1x2.f16x2 d, %4;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]));
  return r;
}
// (x, y) *= f
__device__ __forceinline__ void mul2(float &x, float &y, float f) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(f));
}

__device__ __forceinline__ float e2m1_value(uint32_t nibble) {
  return half_lo(e2m1x2_to_half2(nibble & 0xfu));
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  return half_lo(e4m3x2_to_half2(byte & 0xffu));
}
#endif  // __CUDACC__

}  // namespace d2f
