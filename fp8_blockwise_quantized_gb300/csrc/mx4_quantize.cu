// Quantisation to MXFP4 of activations (rows) and weights (offline).
#include "common.cuh"
#include "kernels.cuh"
#include "mx4.cuh"
#include "ptx.cuh"

namespace gmm {

// Activations: x bf16 [M, K] -> codes [M, K/2], scales [K/128][M] words of the
// four scale bytes of 128 columns.  A half-warp takes one row's 128 columns
// (16 lanes x 16 bytes, four lanes per block of 32); a warp takes the same
// columns of eight consecutive rows, so that its scale words are 32 contiguous
// bytes.  52.8 us at 65536 x 2048, 6.4 TB/s of the 6.8 that a copy reaches (floor
// 50.7).  What bound it was instructions: packed bf16 arithmetic and 32-bit
// indices took it from 65.5 to 59.8 us, one conversion block for the eight codes
// and a path without row checks from there.  Prefetching a warp's next step
// (69.9 us for 65.5), rows of 256 columns a load (66 to 79) and streaming through
// shared memory by bulk copies (69 to 104) were slower.
__global__ void __launch_bounds__(256) mx4_quantize_lhs_kernel(const uint4* __restrict__ x, int M, uint32_t KB,
                                                               uint32_t steps, uint32_t* __restrict__ xq,
                                                               uint32_t* __restrict__ xs) {
  griddep_launch_dependents();
  griddep_wait();  // x may come from the previous kernel
  const int lane = threadIdx.x & 31, half = lane >> 4, l16 = lane & 15;
  const uint32_t nwarps = gridDim.x * 8;
  for (uint32_t st = blockIdx.x * 8 + (threadIdx.x >> 5); st < steps; st += nwarps) {
    const uint32_t mg = st / KB, kb = st - mg * KB;
    const int m0 = static_cast<int>(mg * 8) + half * 4;
    const long long at = (static_cast<long long>(m0) * KB + kb) * 16 + l16;  // 16-byte chunk of x, word of xq
    const uint4* src = x + at;
    uint32_t* dst = xq + at;
    const uint32_t ld = 16 * KB;  // a row of x in 16-byte chunks, and of codes in words
    const int rows = M - m0;      // this half-warp's, when below 4
    uint4 v[4];
    if (rows >= 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __ldcs(src + static_cast<size_t>(i) * ld);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = i < rows ? __ldcs(src + static_cast<size_t>(i) * ld) : make_uint4(0, 0, 0, 0);
    }
    uint32_t bytes = 0;  // this lane's block in the four rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t p[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t m2 = absmax2(absmax2(p[0], p[1]), absmax2(p[2], p[3]));
      m2 = absmax2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
      m2 = absmax2(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
      m2 = absmax2(m2, m2 >> 16);
      const uint32_t b = mx4_scale_byte(m2 & 0xffffu);
      const uint32_t q = mx4_codes8(p, mx4_inverse2(b));
      bytes |= b << (8 * i);
      if (i < rows) dst[static_cast<size_t>(i) * ld] = q;
    }
    // lane i of each half collects row i's word from the four blocks' lanes
    uint32_t word = 0;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint32_t t = __shfl_sync(0xffffffffu, bytes, half * 16 + 4 * g);
      word |= (t >> (8 * (l16 & 3)) & 0xffu) << (8 * g);
    }
    if (l16 < 4 && l16 < rows) xs[static_cast<size_t>(kb) * M + m0 + l16] = word;
  }
}

// Weights: w bf16 [G, K, N] -> codes [G, N, K/2] (K-major), scales
// [G][N/128][K/128] tiles of 512 bytes, the byte of column n and block k/32 at
// (n % 32) * 16 + (n % 128 / 32) * 4 + k / 32 % 4: the 16 bytes of columns l, l +
// 32, l + 64 and l + 96 lie together, which is what lane l of the product's scale
// warps loads at once and stores to tensor memory.  One CTA per 128 x 128 block,
// transposed through shared memory; a thread takes 64 rows (two blocks) of one
// column.  297 us at 256 x 2048 x 1024, 4.6 TB/s (floor 200), once per weight;
// a block's codes are 64 contiguous bytes per column.
__global__ void __launch_bounds__(256) mx4_quantize_rhs_kernel(const uint16_t* __restrict__ w, int K, int N,
                                                               uint8_t* __restrict__ wq, uint8_t* __restrict__ ws) {
  __shared__ uint16_t tile[128][128 + 8];  // [k][n]
  const int NB = N / 128, KB = K / 128;
  const int nb = blockIdx.x % NB, kb = blockIdx.x / NB % KB;
  const long long g = blockIdx.x / (static_cast<long long>(NB) * KB);
  const int t = threadIdx.x;
  {
    const int c = t & 15;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = i * 16 + (t >> 4);
      *reinterpret_cast<uint4*>(&tile[k][8 * c]) = __ldcs(reinterpret_cast<const uint4*>(
          w + (g * K + static_cast<long long>(kb) * 128 + k) * N + static_cast<long long>(nb) * 128 + 8 * c));
    }
  }
  __syncthreads();
  const int n = t >> 1, hk = t & 1;
  uint32_t scales = 0;
  uint4 out[2];
#pragma unroll
  for (int blk = 0; blk < 2; ++blk) {
    const int k0 = 64 * hk + 32 * blk;
    uint32_t p[16];
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      p[i] = tile[k0 + 2 * i][n] | (static_cast<uint32_t>(tile[k0 + 2 * i + 1][n]) << 16);
      m2 = absmax2(m2, p[i]);
    }
    const uint32_t b = mx4_scale_byte(absmax2(m2, m2 >> 16) & 0xffffu);
    const uint32_t inv = mx4_inverse2(b);
    scales |= b << (8 * blk);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t part[4] = {p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]};
      q[i] = mx4_codes8(part, inv);
    }
    out[blk] = make_uint4(q[0], q[1], q[2], q[3]);
  }
  uint4* dst = reinterpret_cast<uint4*>(wq + (g * N + static_cast<long long>(nb) * 128 + n) * (K / 2) +
                                        static_cast<long long>(kb) * 64 + hk * 32);
  dst[0] = out[0];
  dst[1] = out[1];
  uint8_t* sc = ws + ((g * NB + nb) * KB + kb) * 512LL + (n & 31) * 16 + (n >> 5) * 4 + hk * 2;
  *reinterpret_cast<uint16_t*>(sc) = static_cast<uint16_t>(scales);
}

}  // namespace gmm
