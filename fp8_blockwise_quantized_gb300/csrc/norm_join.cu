// The norms before and after a block, joined with its gate and the residual
// stream, and their gradient.
//
//   z = b * rb * w_post,  rb = 1 / sqrt(mean(b^2) + eps)   (z = b without w_post)
//   out = alpha x + beta gate z
//   n = out * ro * w_next,  ro = 1 / sqrt(mean(out^2) + eps)
//
// A CTA takes a row at a time, a thread the same 8 columns of every row, so that the
// sums of the parameters' gradients over the rows stay in its registers, and up to
// 4096 columns (512 threads of 128 registers) the parameters too.  n is rounded
// once, from out before its rounding.
#include "common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace gmm {

namespace {

// Sum over the CTA of two values; red: two buffers in turn, so that one barrier a sum is enough.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2 (*red)[32], int& turn, int warps) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (warps == 1) return make_float2(a, b);
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[turn][threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < warps ? red[turn][lane] : make_float2(0.0f, 0.0f);
  turn ^= 1;
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}

__device__ __forceinline__ float inv_rms(float squares, int K, float eps) {
  return 1.0f / sqrtf(squares / static_cast<float>(K) + eps);
}

// A thread's 8 values of a parameter: from its registers, or where a CTA of NT
// threads has no room for them, from the cache for each row.
template <bool HELD>
struct Param {
  const float* at = nullptr;
  float v[HELD ? 8 : 1];
  __device__ __forceinline__ void set(const float* p, int col) {
    if (!p) return;
    at = p + col;
    if constexpr (HELD) load_params8(at, v);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (HELD) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = v[e];
    } else {
      load_params8(at, f);
    }
  }
};
constexpr int kHeldThreads = 512;

template <typename S, int NT>
__global__ void __launch_bounds__(NT) norm_join_kernel(NormJoinArgs a) {
  __shared__ float2 red[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const int warps = blockDim.x >> 5, col = 8 * threadIdx.x;
  const bool on = col < a.K;
  int turn = 0;
  Param<NT <= kHeldThreads> wp, wn, gc;
  if (on) {
    wp.set(a.w_post, col);
    wn.set(a.w_next, col);
    gc.set(a.gate_col, col);
  }
  const S* x = static_cast<const S*>(a.x);
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const long long at = t * a.K + col;
    typename RawOf<S>::type rx;
    Raw8Bf16 rb, rg;
    if (on) {
      rx.load(x + at);
      if (a.b) rb.load(a.b + at);
      if (a.gate_full) rg.load(a.gate_full + at);
    }
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.0f;
    if (on) rx.get(o);
    if (a.b) {
      float z[8], w[8], scale = 1.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = 0.0f;
      if (on) rb.get(z);
      if (a.w_post) {
        float sq = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(z[e], z[e], sq);
        scale = inv_rms(block_sum2(sq, 0.0f, red, turn, warps).x, a.K, a.eps);
      }
      if (on) {
        if (a.w_post) {
          wp.get(w);
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = z[e] * scale * w[e];
        }
        if (a.gate_full || a.gate_col) {
          if (a.gate_full) rg.get(w); else gc.get(w);
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] *= w[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(a.beta, z[e], a.alpha * o[e]);
        store8(static_cast<S*>(a.out) + at, o);
      }
    }
    if (a.w_next) {
      float sq = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(o[e], o[e], sq);
      const float scale = inv_rms(block_sum2(sq, 0.0f, red, turn, warps).x, a.K, a.eps);
      if (on) {
        float w[8];
        wn.get(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = o[e] * scale * w[e];
        store8(a.n + at, o);
      }
    }
  }
}

// With c = dn * w_next, D = dout + ro c - out ro^3 / K sum(c out); dx = alpha D,
// u = beta D, dgate = u z, and b's gradient from dz = u gate by the same rule.
// A part of the parameters' gradients a CTA, joined by norm_join_reduce_kernel.
template <typename S, int NT>
__global__ void __launch_bounds__(NT) norm_join_bwd_kernel(NormJoinBwdArgs a) {
  __shared__ float2 red[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const int warps = blockDim.x >> 5, col = 8 * threadIdx.x;
  const bool on = col < a.K;
  int turn = 0;
  Param<NT <= kHeldThreads> wp, wn, gc;
  if (on) {
    wp.set(a.w_post, col);
    wn.set(a.w_next, col);
    gc.set(a.gate_col, col);
  }
  float sp[8], sn[8], sg[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sp[e] = sn[e] = sg[e] = 0.0f;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const long long at = t * a.K + col;
    typename RawOf<S>::type ro, rd;
    Raw8Bf16 rb, rn, rg;
    if (on) {
      if (a.dout) rd.load(static_cast<const S*>(a.dout) + at);
      if (a.dn) {
        rn.load(a.dn + at);
        ro.load(static_cast<const S*>(a.out) + at);
      }
      if (a.b) rb.load(a.b + at);
      if (a.gate_full) rg.load(a.gate_full + at);
    }
    float d[8], f[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = 0.0f;
    if (on && a.dout) rd.get(d);
    if (a.dn) {
      float c[8], sq = 0.0f, dot = 0.0f;
      if (on) {
        ro.get(f);
        rn.get(c);
        wn.get(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sq = fmaf(f[e], f[e], sq);
          dot = fmaf(c[e] * w[e], f[e], dot);
        }
      }
      const float2 s = block_sum2(sq, dot, red, turn, warps);
      const float r = inv_rms(s.x, a.K, a.eps), q = s.y * r * r / static_cast<float>(a.K);
      if (on) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sn[e] = fmaf(c[e], f[e] * r, sn[e]);
          d[e] = fmaf(r, fmaf(c[e], w[e], -f[e] * q), d[e]);
        }
      }
    }
    if (on && a.dx) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = a.alpha * d[e];
      store8(static_cast<S*>(a.dx) + at, f);
    }
    if (!a.b) continue;
    // from here d is u = beta D
    float g[8], r = 1.0f, q = 0.0f, sq = 0.0f, dot = 0.0f;
    if (on) {
      rb.get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] *= a.beta;
        g[e] = w[e] = 1.0f;
      }
      if (a.gate_full) rg.get(g);
      if (a.gate_col) gc.get(g);
      if (a.w_post) wp.get(w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sq = fmaf(f[e], f[e], sq);
        dot = fmaf(d[e] * g[e] * w[e], f[e], dot);
      }
    }
    if (a.w_post) {
      const float2 s = block_sum2(sq, dot, red, turn, warps);
      r = inv_rms(s.x, a.K, a.eps);
      q = s.y * r * r / static_cast<float>(a.K);
    }
    if (on) {
      float dg[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float unit = f[e] * r, dz = d[e] * g[e];  // unit: b over its root mean square, or b without w_post
        dg[e] = d[e] * (unit * w[e]);
        sg[e] += dg[e];
        sp[e] = fmaf(dz, unit, sp[e]);
        f[e] = r * fmaf(dz, w[e], -f[e] * q);
      }
      store8(a.db + at, f);
      if (a.gate_full) store8(a.dgate_full + at, dg);
    }
  }
  if (!on) return;
  float* p = a.parts + static_cast<long long>(blockIdx.x) * 3 * a.K + col;
  if (a.dw_post) store8(p, sp);
  if (a.dgate_col) store8(p + a.K, sg);
  if (a.dw_next) store8(p + 2 * a.K, sn);
}

// Sums the CTAs' parts of one parameter's gradient, in their order: 32 columns a
// CTA, 16 warps with every 16th part each.
__global__ void __launch_bounds__(512) norm_join_reduce_kernel(const float* __restrict__ parts, int P, int K,
                                                               float* dw_post, float* dgate, float* dw_next) {
  __shared__ float sums[16][33];
  griddep_launch_dependents();
  griddep_wait();
  float* out = blockIdx.y == 0 ? dw_post : blockIdx.y == 1 ? dgate : dw_next;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (col < K) {
    const float* p = parts + static_cast<long long>(blockIdx.y) * K + col;
#pragma unroll 8
    for (int c = warp; c < P; c += 16) s += p[static_cast<long long>(c) * 3 * K];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < K) {
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) total += sums[w][lane];
    out[col] = total;
  }
}

int row_threads(int64_t K) { return static_cast<int>((K / 8 + 31) / 32 * 32); }

}  // namespace

cudaError_t launch_norm_join(const NormJoinArgs& a, int sms, cudaStream_t stream) {
  const int threads = row_threads(a.K);
  const long long most = static_cast<long long>(sms) * (2048 / threads > 32 ? 32 : 2048 / threads);
  const dim3 grid(static_cast<unsigned>(a.T < most ? a.T : most)), block(threads);
  if (threads <= kHeldThreads)
    return a.f32 ? launch_pdl(norm_join_kernel<float, kHeldThreads>, grid, block, 0, stream, a)
                 : launch_pdl(norm_join_kernel<uint16_t, kHeldThreads>, grid, block, 0, stream, a);
  return a.f32 ? launch_pdl(norm_join_kernel<float, 1024>, grid, block, 0, stream, a)
               : launch_pdl(norm_join_kernel<uint16_t, 1024>, grid, block, 0, stream, a);
}

int norm_join_parts(int64_t T, int64_t K, int sms) {
  const int threads = row_threads(K);
  const long long most = static_cast<long long>(sms) * (threads > 512 ? 1 : 512 / threads);
  return static_cast<int>(T < most ? T : most);
}

cudaError_t launch_norm_join_bwd(const NormJoinBwdArgs& a, int sms, cudaStream_t stream) {
  const int threads = row_threads(a.K), parts = norm_join_parts(a.T, a.K, sms);
  const dim3 grid(parts), block(threads);
  cudaError_t e = cudaSuccess;
  if (parts > 0) {
    if (threads <= kHeldThreads)
      e = a.f32 ? launch_pdl(norm_join_bwd_kernel<float, kHeldThreads>, grid, block, 0, stream, a)
                : launch_pdl(norm_join_bwd_kernel<uint16_t, kHeldThreads>, grid, block, 0, stream, a);
    else
      e = a.f32 ? launch_pdl(norm_join_bwd_kernel<float, 1024>, grid, block, 0, stream, a)
                : launch_pdl(norm_join_bwd_kernel<uint16_t, 1024>, grid, block, 0, stream, a);
  }
  if (e != cudaSuccess || !(a.dw_post || a.dgate_col || a.dw_next)) return e;
  return launch_pdl(norm_join_reduce_kernel, dim3(static_cast<unsigned>((a.K + 31) / 32), 3), dim3(512), 0, stream,
                    static_cast<const float*>(a.parts), parts, static_cast<int>(a.K), a.dw_post, a.dgate_col, a.dw_next);
}

}  // namespace gmm
