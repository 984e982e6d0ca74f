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

}  // namespace pkv
