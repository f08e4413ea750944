// MXFP4 arithmetic shared by the quantising kernels and the fused epilogue:
// blocks of 32 values share a power-of-two scale 2^(b - 127) (E8M0 byte b) and
// each value is an E2M1 code.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace gmm {

// The scale byte of a block from the largest |value|'s bf16 bits:
// floor(log2(absmax)) - 2, 2 being E2M1's largest exponent, on the biased
// exponent field E: max(E - 2, 0).  Zero and subnormal absmax give 0
// (2^-127); a block that holds an infinity or NaN (E = 255) gets 255, NaN.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t absmax_bits) {
  const uint32_t e = absmax_bits >> 7;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 1 / scale, exact for every scale byte of finite values (0 .. 252)
__device__ __forceinline__ float mx4_inverse(uint32_t byte) {
  return __uint_as_float((254u - (byte > 253u ? 253u : byte)) << 23);
}
// max of |bf16| over a pair of packed pairs, each half on its own
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
  return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu);
}
// 8 bf16 values times `inv` -> 8 E2M1 codes, the first in the lowest 4 bits;
// nearest, ties to even, saturating at 6.  The product is exact (a power of two).
__device__ __forceinline__ uint32_t mx4_codes8(const uint32_t (&p)[4], float inv) {
  uint32_t q = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = make_float2(__uint_as_float(p[i] << 16) * inv, __uint_as_float(p[i] & 0xffff0000u) * inv);
    q |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(v, __NV_E2M1, cudaRoundNearest)) << (8 * i);
  }
  return q;
}

}  // namespace gmm
