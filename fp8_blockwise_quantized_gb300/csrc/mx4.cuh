// MXFP4 arithmetic shared by the quantising kernels and the fused epilogue:
// blocks of 32 values share a power-of-two scale 2^(b - 127) (E8M0 byte b) and
// each value is an E2M1 code.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace gmm {

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t v) {
  return *reinterpret_cast<const __nv_bfloat162*>(&v);
}
__device__ __forceinline__ uint32_t as_bits(const __nv_bfloat162& v) {
  return *reinterpret_cast<const uint32_t*>(&v);
}

// max of |bf16| over two packed pairs, each half on its own (NaN stays NaN)
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
  return as_bits(__hmax2_nan(__habs2(as_bf162(a)), __habs2(as_bf162(b))));
}
// The scale byte of a block from the largest |value|'s bf16 bits:
// floor(log2(absmax)) - 2, 2 being E2M1's largest exponent, on the biased
// exponent field E: max(E - 2, 0).  Zero and subnormal absmax give 0
// (2^-127); a block that holds an infinity or NaN (E = 255) gets 255, NaN.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t absmax_bits) {
  const uint32_t e = absmax_bits >> 7;
  return e == 255u ? 255u : max(e, 2u) - 2u;
}
// 1 / scale in both halves of a bf16 pair, exact for every scale byte of finite
// values (0 .. 252)
__device__ __forceinline__ uint32_t mx4_inverse2(uint32_t byte) { return (254u - min(byte, 253u)) * 0x00800080u; }
// 8 bf16 values / scale -> 8 E2M1 codes, the first in the lowest 4 bits;
// nearest, ties to even, saturating at 6.  The quotient is a bf16 product with
// a power of two: exact, or too small for any code but 0.
__device__ __forceinline__ uint32_t mx4_codes8(const uint32_t (&p)[4], uint32_t inv2) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t s = as_bits(__hmul2(as_bf162(p[i]), as_bf162(inv2)));
    v[2 * i] = __uint_as_float(s << 16);
    v[2 * i + 1] = __uint_as_float(s & 0xffff0000u);
  }
  // cvt's first source goes to the upper code of the pair
  uint32_t q;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(q)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return q;
}

}  // namespace gmm
