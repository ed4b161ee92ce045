// fp4.cuh — the element types of the 4-bit paged cache: 4-bit floats (e2m1) in
// groups of 16 with an 8-bit scale (e4m3).  A code times a scale has at most
// six significant bits and lies in [2^-10, 2688] (or is 0), so it is exact in
// fp16, and in every wider type.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gb300 {
namespace fp4 {

// The codes of a word's four bytes as fp16 pairs (low half: the low code).  The
// split into 8-bit registers is one move; every byte at every place is tested
// in each kernel that splits so, since the join that mirrors it is compiled
// wrongly (codes_of).  With a shift and a narrowing for each byte instead, 8 x
// 32768 single keys take 84.7 us instead of 75.4, 4096 tokens over 32768 keys
// 1505 instead of 1450.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
// Two scales (the low 16 bits of w) as an fp16 pair.
__device__ __forceinline__ uint32_t scales_f16(uint32_t w) {
  uint32_t o;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}"
      : "=r"(o)
      : "r"(w));
  return o;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) {
  return *reinterpret_cast<__half2*>(&x);
}
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Scale byte of a group whose largest magnitude is `top`: top / 6 rounded to
// e4m3 within [2^-9, 448], and its value.
__device__ __forceinline__ uint32_t scale_of(float top, float* value) {
  uint32_t s;
  asm("{\n\t.reg .b16 x;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.u32.u16 %0, x;\n\t}"
      : "=r"(s)
      : "f"(__fdiv_rn(top, 6.f)), "f"(0.f));
  s &= 0xffu;
  if (s == 0) s = 1;  // 2^-9, the least
  *value = __low2float(as_half2(scales_f16(s)));
  return s;
}
// Eight numbers as codes, ties to even, at most 6 in magnitude: a word, the
// first in its low four bits.  (Each byte through a register of its own: joined
// as 8-bit registers in one move, the first two come out wrong in the appends,
// whatever the data, nvcc 13.0.88.)
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8]) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b8 c;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\t"
        "cvt.u32.u8 %0, c;\n\t}"
        : "=r"(b[i])
        : "f"(x[2 * i]), "f"(x[2 * i + 1]));
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

}  // namespace fp4
}  // namespace gb300
