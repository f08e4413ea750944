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
  uint32_t q = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t s = as_bits(__hmul2(as_bf162(p[i]), as_bf162(inv2)));
    const float2 v = make_float2(__uint_as_float(s << 16), __uint_as_float(s & 0xffff0000u));
    q |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(v, __NV_E2M1, cudaRoundNearest)) << (8 * i);
  }
  return q;
}

}  // namespace gmm
