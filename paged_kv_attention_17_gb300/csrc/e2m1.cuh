// The 4-bit cache format: E2M1 codes with one E4M3 scale per 16 elements.
//
// K and V are one tensor of pages each, [num_blocks][num_kv_heads][9 D bytes].
// The page of one (block, KV head) is 16 token rows of D / 2 code bytes
// (element 2 i in the low nibble of byte i), then 16 token rows of D / 16
// scale bytes, so a block of one head is one contiguous run of 1152 (D 128) or
// 576 (D 64) bytes, and moving a page moves its scales.  An element stands for
//   t * value(scale) * value(code)
// with t the tensor's fp32 scale.  value(scale) * value(code) has at most six
// significant bits and a magnitude of 0 or 2^-10 .. 2688, so it is a bf16
// value and a normal f16 value: widening to either is exact.
#pragma once

#include "common.cuh"

namespace pkv {

constexpr int kQuant = 16;                               // elements per scale
template <int D>
struct E2m1Page {
  static constexpr int kRowCodes = D / 2;                // code bytes of a token row
  static constexpr int kRowScales = D / kQuant;          // scale bytes of a token row
  static constexpr int kCodes = kBlock * kRowCodes;
  static constexpr int kScales = kBlock * kRowScales;
  static constexpr int kBytes = kCodes + kScales;        // 9 D
};

// Eight E2M1 codes (a word, element 0 in the low nibble) -> four f16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\tmov.b32 {c0, c1, c2, c3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, c0;\n\tcvt.rn.f16x2.e2m1x2 %1, c1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c2;\n\tcvt.rn.f16x2.e2m1x2 %3, c3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Two E4M3 codes (low 16 bits, element 0 in the low byte) -> an f16 pair.
__device__ __forceinline__ uint32_t scales2_to_f16x2(uint32_t two_codes) {
  uint32_t h2;
  asm("{\n\t.reg .b16 c, u;\n\tmov.b32 {c, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}"
      : "=r"(h2)
      : "r"(two_codes));
  return h2;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t byte_perm(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// ---------------------------------------------------------------------------
// Quantising one block: 16 elements x of a row, divided by the tensor's scale t,
//   y = RN32(x / t),  s = E4M3(RN32(max |y| / 6)),  code = E2M1(RN32(y / s)).
// ---------------------------------------------------------------------------

// Quotients by a fixed t.  With inv = RN32(1 / t), q = RN32(x inv) is within two
// ulps of x / t, and each step q - inv (q t - x) with one rounding an operation
// takes its error to the square; the last step from a q within one ulp is the
// correctly rounded quotient (Markstein's theorem; P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).  For t in
// [2^-40, 2^40] no operation of it underflows where y matters: |y| < 2^-60 is a
// code 0 whatever its last bit.  Taking the remainder as q t - x keeps the sign
// of a zero x.  Blocks with a y beyond 1e30, an infinity or a NaN are left to the
// plain division.
struct Divisor {
  float t, inv;
  bool plain;
};
__device__ __forceinline__ Divisor divisor(float t) {
  return {t, __fdiv_rn(1.f, t), !(t >= 0x1p-40f && t <= 0x1p40f)};
}
__device__ __forceinline__ float quotient_step(float q, float x, float t, float inv) {
  return fmaf(-fmaf(q, t, -x), inv, q);
}
// max(a, |b|), NaN if either is
__device__ __forceinline__ float max_abs_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
  return d;
}

// A block's 16 inputs as floats.
__device__ __forceinline__ void load16(const float* p, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(p) + i);
    f[4 * i] = v.x;
    f[4 * i + 1] = v.y;
    f[4 * i + 2] = v.z;
    f[4 * i + 3] = v.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    f[8 * i] = bf16_lo(w.x);
    f[8 * i + 1] = bf16_hi(w.x);
    f[8 * i + 2] = bf16_lo(w.y);
    f[8 * i + 3] = bf16_hi(w.y);
    f[8 * i + 4] = bf16_lo(w.z);
    f[8 * i + 5] = bf16_hi(w.z);
    f[8 * i + 6] = bf16_lo(w.w);
    f[8 * i + 7] = bf16_hi(w.w);
  }
}

// (a, b) -> two E2M1 codes, a in the low nibble
__device__ __forceinline__ uint32_t float2_to_e2m1x2(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\tcvt.u32.u8 %0, c;\n\t}"
      : "=r"(r)
      : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ void quantise16(const float (&x)[16], const Divisor& d, uint2& codes,
                                           uint32_t& scale) {
  float y[16];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float q = quotient_step(x[i] * d.inv, x[i], d.t, d.inv);
    y[i] = quotient_step(q, x[i], d.t, d.inv);
    a = max_abs_nan(a, y[i]);
  }
  const bool plain = d.plain || !(a <= 1e30f);
  if (plain) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      y[i] = __fdiv_rn(x[i], d.t);
      a = max_abs_nan(a, y[i]);
    }
  }
  codes = make_uint2(0, 0);
  scale = 0x7F;                                          // a NaN among the 16: its block's scale
  if (a != a) return;
  scale = float2_to_e4m3x2(__fdiv_rn(a, 6.f), 0.f) & 0xFFu;
  if (scale == 0) return;
  // Quotients by s, of four significant bits: y / s is at least 2^-29 (relative)
  // from every midpoint of two floats, so one step, whose error before its last
  // rounding is about 2^-46, rounds correctly.
  const float s = e4m3x2_to_float2(scale).x, inv = __fdiv_rn(1.f, s);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y0 = y[2 * i], y1 = y[2 * i + 1];
    const float z0 = plain ? __fdiv_rn(y0, s) : quotient_step(y0 * inv, y0, s, inv);
    const float z1 = plain ? __fdiv_rn(y1, s) : quotient_step(y1 * inv, y1, s, inv);
    c[i] = float2_to_e2m1x2(z0, z1);
  }
  codes = make_uint2(c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24),
                     c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24));
}

}  // namespace pkv
