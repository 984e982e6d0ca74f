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
#include "e2m1_index.h"

namespace pkv {

static_assert(kPageTokens == kBlock, "a page is a cache block");

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
// of a zero x.  Other t, and blocks with a y beyond 1e30, an infinity or a NaN,
// are left to the plain division.
struct Divisor {
  float t, inv;                                          // inv: RN32(1 / t)
};
__device__ __forceinline__ float quotient_step(float q, float x, float t, float inv) {
  return fmaf(-fmaf(q, t, -x), inv, q);
}
// The same on two quotients (-x) / t at once: from q0 = x ninv, ninv = -inv, each
// step is q + (q t + x) ninv.  (Negated, so that no operand is: a second division
// of the negative quotient has the sign of x again.)
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 halves(Pair v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ Pair pair_mul(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair pair_fma(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ Pair quotient_step(Pair q, Pair x, Pair t, Pair ninv) {
  return pair_fma(pair_fma(q, t, x), ninv, q);
}
// max(a, |b|, |c|), NaN if any is
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}

// A block's 16 inputs, as loaded and as floats.
template <typename S>
struct Raw16 {
  uint4 w[static_cast<int>(sizeof(S))];
  __device__ __forceinline__ void load(const S* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(S)); ++i)
      w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void floats(float (&f)[16]) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(S)); ++i) {
      const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(S) == 4) {
          f[4 * i + k] = __uint_as_float(v[k]);
        } else {
          f[8 * i + 2 * k] = bf16_lo(v[k]);
          f[8 * i + 2 * k + 1] = bf16_hi(v[k]);
        }
      }
    }
  }
  // The largest magnitude (an infinity or a NaN counts as the larger, by its bits).
  __device__ __forceinline__ float largest() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(S)); ++i) {
      const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        m = sizeof(S) == 4 ? max(m, v[k] & 0x7FFFFFFFu) : __vmaxu2(m, v[k] & 0x7FFF7FFFu);
    }
    return __uint_as_float(sizeof(S) == 4 ? m : max(m << 16, m & 0xFFFF0000u));
  }
};

// (a, b) -> two E2M1 codes, a in the low nibble
__device__ __forceinline__ uint32_t float2_to_e2m1x2(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\tcvt.u32.u8 %0, c;\n\t}"
      : "=r"(r)
      : "f"(b), "f"(a));
  return r;
}

// Eight values -> eight codes, the first in the low nibble.
__device__ __forceinline__ uint32_t floats_to_e2m1x8(float2 a, float2 b, float2 c, float2 d) {
  uint32_t r;
  asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n\t"
      "mov.b32 %0, {c0, c1, c2, c3};\n\t}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return r;
}

// The definition with plain divisions (a call: rare, and kept out of the
// registers of the common path).
static __device__ __noinline__ uint3 quantise16_plain(const float* x, float t) {
  float a = 0.f;
  for (int i = 0; i < 16; i += 2)
    a = max_abs_nan(a, __fdiv_rn(x[i], t), __fdiv_rn(x[i + 1], t));
  if (a != a) return make_uint3(0, 0, 0x7F);             // a NaN among the 16
  const uint32_t scale = float2_to_e4m3x2(__fdiv_rn(a, 6.f), 0.f) & 0xFFu;
  uint32_t c[2] = {0, 0};
  const float s = e4m3x2_to_float2(scale).x;
  for (int i = 0; i < 16 && scale != 0; i += 2)
    c[i / 8] |= float2_to_e2m1x2(__fdiv_rn(__fdiv_rn(x[i], t), s),
                                 __fdiv_rn(__fdiv_rn(x[i + 1], t), s))
                << (4 * (i % 8));
  return make_uint3(c[0], c[1], scale);
}

template <typename S>
__device__ __forceinline__ void quantise16(const Raw16<S>& raw, const Divisor& d, uint2& codes,
                                           uint32_t& scale) {
  float x[16];
  raw.floats(x);
  // max |RN(x / t)| = RN(max |x| / t): rounding is monotonic
  const float top = raw.largest();
  const float a = quotient_step(quotient_step(top * d.inv, top, d.t, d.inv), top, d.t, d.inv);
  if (!(a <= 1e30f) || !(d.t >= 0x1p-40f && d.t <= 0x1p40f)) {
    float copy[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) copy[i] = x[i];
    const uint3 r = quantise16_plain(copy, d.t);
    codes = make_uint2(r.x, r.y);
    scale = r.z;
    return;
  }
  // Quotients by 6 and by s, divisors of at most four significant bits: such a
  // quotient is at least 2^-29 (relative) from every midpoint of two floats, so
  // one step, whose error before its last rounding is below 2^-43 even from an
  // approximate reciprocal (2^-22), rounds correctly.
  constexpr float kInv6 = 1.f / 6.f;
  scale = float2_to_e4m3x2(quotient_step(a * kInv6, a, 6.f, kInv6), 0.f) & 0xFFu;
  codes = make_uint2(0, 0);
  if (scale == 0) return;
  const float s = e4m3x2_to_float2(scale).x;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const Pair t2 = pair_of(d.t, d.t), ninv2 = pair_of(-d.inv, -d.inv);
  const Pair s2 = pair_of(s, s), nis2 = pair_of(-inv, -inv);
  float2 z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const Pair x2 = pair_of(x[2 * i], x[2 * i + 1]);
    Pair y = quotient_step(pair_mul(x2, ninv2), x2, t2, ninv2);   // -y, in the end
    y = quotient_step(y, x2, t2, ninv2);
    z[i] = halves(quotient_step(pair_mul(y, nis2), y, s2, nis2));
  }
  codes = make_uint2(floats_to_e2m1x8(z[0], z[1], z[2], z[3]),
                     floats_to_e2m1x8(z[4], z[5], z[6], z[7]));
}

}  // namespace pkv
