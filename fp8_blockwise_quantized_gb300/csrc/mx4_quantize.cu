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
// bytes, with all loads issued before the first is used.
__global__ void __launch_bounds__(256) mx4_quantize_lhs_kernel(const uint4* __restrict__ x, int M, int KB,
                                                               uint32_t* __restrict__ xq, uint32_t* __restrict__ xs) {
  griddep_launch_dependents();
  griddep_wait();  // x may come from the previous kernel
  const int lane = threadIdx.x & 31, half = lane >> 4, l16 = lane & 15;
  const long long warp_id = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const long long nwarps = (static_cast<long long>(gridDim.x) * blockDim.x) >> 5;
  const long long steps = (M + 7) / 8 * static_cast<long long>(KB);
  for (long long st = warp_id; st < steps; st += nwarps) {
    const long long m0 = st / KB * 8 + half * 4, kb = st % KB;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = m0 + i < M ? __ldcs(x + ((m0 + i) * KB + kb) * 16 + l16) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t p[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t m2 = absmax2(absmax2(p[0], p[1]), absmax2(p[2], p[3]));
      m2 = max(m2 & 0xffffu, m2 >> 16);
      m2 = max(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
      m2 = max(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
      const uint32_t b = mx4_scale_byte(m2);
      const uint32_t q = mx4_codes8(p, mx4_inverse(b));
      uint32_t word = b << (8 * (l16 >> 2));
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
      word |= __shfl_xor_sync(0xffffffffu, word, 8);
      if (m0 + i < M) {
        xq[((m0 + i) * KB + kb) * 16 + l16] = q;
        if (l16 == 0) xs[kb * M + m0 + i] = word;
      }
    }
  }
}

// Weights: w bf16 [G, K, N] -> codes [G, N, K/2] (K-major), scales
// [G][N/128][K/128] tiles of 512 bytes, the byte of column n and block k/32 at
// (n % 32) * 16 + (n % 128 / 32) * 4 + k / 32 % 4: the order in which one copy
// puts a tile into tensor memory.  One CTA per 128 x 128 block, transposed
// through shared memory; a thread takes 64 rows (two blocks) of one column.
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
    const uint32_t b = mx4_scale_byte(max(m2 & 0xffffu, m2 >> 16));
    const float inv = mx4_inverse(b);
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
