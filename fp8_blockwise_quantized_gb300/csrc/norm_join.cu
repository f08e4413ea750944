// The norms before and after a block, joined with its gate and the residual
// stream, and their gradient.
//
//   z = b * rb * w_post,  rb = 1 / sqrt(mean(b^2) + eps)   (z = b without w_post)
//   out = alpha x + beta gate z
//   n = out * ro * w_next,  ro = 1 / sqrt(mean(out^2) + eps)
//
// A thread takes the same columns of every row it takes, so that what is constant in a
// column (beta, w_post, a gate per column: one factor) and the sums of the parameters'
// gradients over the rows stay in its registers.  n is rounded once, from out before
// its rounding.
//
// Bound by HBM, with the instructions close behind: two columns an instruction, sums
// of two values for five exchanges, loads without predicates.  At 8192 x 2048 (floor
// at the measured copy rate in brackets): forward 20.9 us (20.1) with a bf16 stream,
// 33.5 (30.2) with an fp32 stream and a gate per column; backward 39.4 (30.2) and 52.6
// (45.2), 5 of them the sums over the rows.  The next row's values are on their way to
// registers while a row is worked on: through shared memory (asynchronous copies, two
// to six rows ahead) they pass the SM's load path twice, and the same calls took 22.0,
// 40.2, 42.1 and 71.4 us; rows asked for in the L2 further ahead, 22.6 to 25.6 and
// 36.0 to 40.8 us forward.
#include "common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace gmm {

namespace {

// 8 columns, and arithmetic on pairs of them (one instruction a pair).
struct Cols {
  float2 v[4];
  __device__ __forceinline__ static Cols of(float f) {
    Cols c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c.v[i] = make_float2(f, f);
    return c;
  }
};
__device__ __forceinline__ Cols operator*(const Cols& a, const Cols& b) {
  Cols c;
#pragma unroll
  for (int i = 0; i < 4; ++i) c.v[i] = __fmul2_rn(a.v[i], b.v[i]);
  return c;
}
__device__ __forceinline__ Cols operator*(const Cols& a, float f) {
  Cols c;
#pragma unroll
  for (int i = 0; i < 4; ++i) c.v[i] = __fmul2_rn(a.v[i], make_float2(f, f));
  return c;
}
__device__ __forceinline__ Cols fma8(const Cols& a, const Cols& b, const Cols& c) {
  Cols r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __ffma2_rn(a.v[i], b.v[i], c.v[i]);
  return r;
}
__device__ __forceinline__ Cols fma8(const Cols& a, float f, const Cols& c) {
  Cols r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __ffma2_rn(a.v[i], make_float2(f, f), c.v[i]);
  return r;
}
// sum of a * b over the 8 columns
__device__ __forceinline__ float dot8(const Cols& a, const Cols& b) {
  float2 s = __fmul2_rn(a.v[0], b.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = __ffma2_rn(a.v[i], b.v[i], s);
  return s.x + s.y;
}
__device__ __forceinline__ Cols cols_of(const float4& a, const float4& b) {
  Cols c;
  c.v[0] = make_float2(a.x, a.y), c.v[1] = make_float2(a.z, a.w);
  c.v[2] = make_float2(b.x, b.y), c.v[3] = make_float2(b.z, b.w);
  return c;
}
__device__ __forceinline__ Cols cols_of(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  Cols c;
#pragma unroll
  for (int i = 0; i < 4; ++i) c.v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return c;
}

// Where a thread stands: its row among the CTA's, its columns, its row's warps.
struct Place {
  int team, rows, col, warps, warp;
  __device__ __forceinline__ explicit Place(int row_threads) {
    team = threadIdx.x / row_threads;
    rows = blockDim.x / row_threads;
    const int in_row = threadIdx.x - team * row_threads;
    col = 8 * in_row;
    warp = in_row >> 5;
    warps = row_threads >> 5;
  }
};

// N sums (1 or 2) over a row's threads.  Of two, neighbours 16 lanes apart exchange one
// each, so that the lower half of a warp goes on with the first and the upper half with
// the second.  The warps' sums lie in 32 words a row, 32 / N a value; every warp adds
// them up, a lane a word.  red: two buffers in turn, so that one barrier is enough;
// zeros where no warp writes.
constexpr int kMaxTeams = 8;
using SumBuffer = float[2][kMaxTeams + 1][32];
template <int N>
struct Sums {
  float (*red)[kMaxTeams + 1][32];
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&s)[N], const Place& p) {
    constexpr int kSpan = 32 / N;
    const int lane = threadIdx.x & 31;
    float v = s[0];
    if constexpr (N == 2) {
      const bool up = lane & 16;
      v = (up ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, up ? s[0] : s[1], 16);
    }
#pragma unroll
    for (int d = kSpan / 2; d >= 1; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (p.warps > 1) {
      float* row = red[turn][p.team];
      if ((lane & (kSpan - 1)) == 0) row[lane + p.warp] = v;
      __syncthreads();
      turn ^= 1;
      v = row[lane];
      if (p.warps > 8) v += __shfl_xor_sync(0xffffffffu, v, 8);
      if (p.warps > 4) v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      v += __shfl_xor_sync(0xffffffffu, v, 1);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = __shfl_sync(0xffffffffu, v, kSpan * i);
  }
};
// Zeros for a kernel's buffers.
__device__ __forceinline__ void clear(SumBuffer& red) {
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(red) / sizeof(float)); i += blockDim.x)
    (&red[0][0][0])[i] = 0.0f;
  __syncthreads();
}

// Eight columns as they lie in memory.
template <typename S>
struct Raw;
template <>
struct Raw<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ Cols get() const { return cols_of(v); }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ Cols get() const { return cols_of(a, b); }
};
__device__ __forceinline__ void put8(uint16_t* p, const Cols& c) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(c.v[0].x, c.v[0].y), pack_bf16x2(c.v[1].x, c.v[1].y),
                                            pack_bf16x2(c.v[2].x, c.v[2].y), pack_bf16x2(c.v[3].x, c.v[3].y));
}
__device__ __forceinline__ void put8(float* p, const Cols& c) {
  reinterpret_cast<float4*>(p)[0] = make_float4(c.v[0].x, c.v[0].y, c.v[1].x, c.v[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(c.v[2].x, c.v[2].y, c.v[3].x, c.v[3].y);
}

// factor * p * q of 8 columns (a null pointer counts as 1).
__device__ __forceinline__ Cols factors8(const float* p, const float* q, float factor, int col) {
  Cols c = Cols::of(factor);
  auto at = [&](const float* f) {
    const float4* v = reinterpret_cast<const float4*>(f + col);
    return cols_of(__ldg(v), __ldg(v + 1));
  };
  if (p) c = c * at(p);
  if (q) c = c * at(q);
  return c;
}

// rsqrt is within 2 units of the last place.
__device__ __forceinline__ float inv_rms(float squares, float inv_k, float eps) {
  return rsqrtf(fmaf(squares, inv_k, eps));
}

// V vectors of 8 columns a thread, at most NT threads a CTA.  A thread without columns
// reads those of others and adds nothing; the row ahead of the last is the last again.
template <typename S, int V, int NT, bool FULL>
__global__ void __launch_bounds__(NT, 512 / NT) norm_join_kernel(NormJoinArgs a) {
  __shared__ SumBuffer red;
  griddep_launch_dependents();
  clear(red);
  const Place me(a.row_threads);
  griddep_wait();
  const long long step = static_cast<long long>(gridDim.x) * me.rows;
  const float inv_k = 1.0f / static_cast<float>(a.K);
  bool on[V];
  int col[V];
  Cols pw[V], wn[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = me.col + 8 * a.row_threads * v;
    on[v] = me.team < me.rows && col[v] < a.K;
    if (!on[v]) col[v] = 0;
    pw[v] = factors8(a.w_post, a.gate_col, a.beta, col[v]);
    wn[v] = factors8(a.w_next, nullptr, 1.0f, col[v]);
  }
  Raw<S> x[V];
  Raw<uint16_t> b[V], g[V];
  auto fetch = [&](long long t) {
    const long long at = (t < a.T ? t : a.T - 1) * a.K;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v].load(static_cast<const S*>(a.x) + at + col[v]);
      if (a.b) b[v].load(a.b + at + col[v]);
      if (FULL) g[v].load(a.gate_full + at + col[v]);
    }
  };
  long long t = static_cast<long long>(blockIdx.x) * me.rows + me.team;
  fetch(t);
  Sums<1> sums{red};
  for (long long t0 = t - me.team; t0 < a.T; t0 += step, t += step) {
    const long long at = t * a.K;
    Cols o[V], z[V];
    float s[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = x[v].get() * a.alpha;
    if (a.b) {
      float r = 1.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        z[v] = b[v].get();
        if (on[v]) s[0] += dot8(z[v], z[v]);
        z[v] = z[v] * pw[v];
        if (FULL) z[v] = z[v] * g[v].get();
      }
      fetch(t + step);
      if (a.w_post) {
        sums(s, me);
        r = inv_rms(s[0], inv_k, a.eps);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        o[v] = fma8(z[v], r, o[v]);
        if (on[v] && t < a.T) put8(static_cast<S*>(a.out) + at + col[v], o[v]);
      }
    } else {
      fetch(t + step);
    }
    if (a.w_next) {
      s[0] = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (on[v]) s[0] += dot8(o[v], o[v]);
      sums(s, me);
      const float r = inv_rms(s[0], inv_k, a.eps);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (on[v] && t < a.T) put8(a.n + at + col[v], o[v] * r * wn[v]);
    }
  }
}

constexpr int kOneCtas = 8;

// The parameters' gradients of column c from its two sums.
__device__ __forceinline__ void put_columns(const NormJoinBwdArgs& a, int c, float post, float next) {
  if (a.dw_post) a.dw_post[c] = a.beta * post * (a.gate_col ? a.gate_col[c] : 1.0f);
  if (a.dgate_col) a.dgate_col[c] = a.beta * post * (a.w_post ? a.w_post[c] : 1.0f);
  if (a.dw_next) a.dw_next[c] = next;
}

// With c = dn * w_next, D = dout + ro (c - out ro^2 / K sum(c out)); dx = alpha D.
// With p = beta * w_post * gate, b's gradient is that of its norm from t = D p:
// db = rb (t - b rb^2 / K sum(t b)).  (A cube of ro or rb leaves fp32's range where the
// gradient does not: rows below 1e-13 with eps = 0.)  With s = sum over the rows of
// D b rb (times a gate per element), dw_post = beta gate s and a column gate's gradient
// beta w_post s: one sum for both, a part of it a CTA (and of dw_next's), joined by
// norm_join_reduce_kernel.
//
// V = 2 (over 4096 columns): the registers hold the sums and the factors, but not the
// row ahead, which goes through shared memory, and its values are read there again when
// they are needed again.  2048 x 8192: 41.8 us with a bf16 stream (floor 30.2), 56.3
// with fp32 (45.2); with the row read when its turn came, asked for in the L2 before,
// and factors from the cache, 55.0 and 79.4.  What is left is a row's two sums, one after
// the other, with no other row in the SM.
// ONE: few rows are one cluster's, whose CTAs add up each other's sums; no parts and no
// second kernel.
template <typename S, int V, int NT, bool FULL, bool ONE>
__global__ void __launch_bounds__(NT, 512 / NT) norm_join_bwd_kernel(NormJoinBwdArgs a) {
  static_assert(V == 1 || !ONE, "a thread's columns are 8 words of shared memory a sum");
  constexpr bool kHeld = V == 1;
  constexpr int kS = sizeof(S) / 2, kChunks = V * (2 * kS + 2 + FULL);  // 16 bytes of a row
  extern __shared__ uint4 ahead[];                                      // [2][kChunks][NT] where V = 2
  __shared__ SumBuffer red;
  griddep_launch_dependents();
  clear(red);
  const Place me(a.row_threads);
  griddep_wait();
  const long long step = static_cast<long long>(gridDim.x) * me.rows;
  const float inv_k = 1.0f / static_cast<float>(a.K);
  bool on[V];
  int col[V];
  Cols post[V], next[V], sb[V], sn[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = me.col + 8 * a.row_threads * v;
    on[v] = me.team < me.rows && col[v] < a.K;
    if (!on[v]) col[v] = 0;
    sb[v] = sn[v] = Cols::of(0.0f);
    post[v] = factors8(a.w_post, a.gate_col, a.beta, col[v]);
    next[v] = factors8(a.w_next, nullptr, 1.0f, col[v]);
  }
  Raw<S> rd[V], ro[V];
  Raw<uint16_t> rn[V], rb[V], rg[V];
  auto fetch = [&](long long t) {
    const long long row = (t < a.T ? t : a.T - 1) * a.K;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const long long at = row + col[v];
      if (a.dout) rd[v].load(static_cast<const S*>(a.dout) + at);
      if (a.dn) {
        rn[v].load(a.dn + at);
        ro[v].load(static_cast<const S*>(a.out) + at);
      }
      if (a.b) rb[v].load(a.b + at);
      if (FULL) rg[v].load(a.gate_full + at);
    }
  };
  // Through shared memory each warp copies its own columns as they lie in memory: of
  // fp32 a lane takes every 32nd 16 bytes and reads two neighbours (with its own 32 bytes
  // in two copies every sector was read twice: 75.2 us).
  const int lane = threadIdx.x & 31;
  int turn = 0;
  auto stage = [&](long long t) {
    if (t < a.T) {
      const long long row = t * a.K;
      uint4* to = ahead + turn * kChunks * NT + threadIdx.x;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (kS == 2) {
          const int first = me.col + 8 * (a.row_threads * v - lane) + 4 * lane;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int at = first + 128 * i;
            uint4* here = to + 2 * v * NT + (threadIdx.x - lane) + 32 * i;
            if (me.team >= me.rows || at >= a.K) continue;
            if (a.dout) cp_async_16(here, static_cast<const S*>(a.dout) + row + at);
            if (a.dn) cp_async_16(here + 2 * V * NT, static_cast<const S*>(a.out) + row + at);
          }
        }
        if (!on[v]) continue;
        if constexpr (kS == 1) {
          if (a.dout) cp_async_16(to + v * NT, static_cast<const S*>(a.dout) + row + col[v]);
          if (a.dn) cp_async_16(to + (V + v) * NT, static_cast<const S*>(a.out) + row + col[v]);
        }
        if (a.dn) cp_async_16(to + (2 * kS * V + v) * NT, a.dn + row + col[v]);
        if (a.b) cp_async_16(to + (2 * kS * V + V + v) * NT, a.b + row + col[v]);
        if (FULL) cp_async_16(to + (2 * kS * V + 2 * V + v) * NT, a.gate_full + row + col[v]);
      }
    }
    cp_async_commit();
    turn ^= 1;
  };
  const uint4* at_hand = nullptr;
  auto wide = [&](int i) {
    if constexpr (kS == 1) return cols_of(at_hand[i * NT]);
    // lanes 4 to 7 of 8 read their second 16 bytes first: no two in one bank
    const bool swap = lane & 4;
    const float4* q = reinterpret_cast<const float4*>(at_hand + 2 * i * NT + threadIdx.x);
    const float4 x = q[swap], y = q[!swap];
    return cols_of(swap ? y : x, swap ? x : y);
  };
  auto half = [&](int i) { return cols_of(at_hand[(2 * kS * V + i) * NT]); };
#pragma unroll
  for (int v = 0; v < V; ++v) rd[v].zero();
  long long t = static_cast<long long>(blockIdx.x) * me.rows + me.team;
  if (kHeld)
    fetch(t);
  else
    stage(t);
  Sums<2> sums{red};
  for (long long t0 = t - me.team; t0 < a.T; t0 += step, t += step) {
    const long long row = t * a.K;
    if constexpr (!kHeld) {
      __syncthreads();  // the row that the next one replaces has been read
      at_hand = ahead + (turn ^ 1) * kChunks * NT + threadIdx.x;
      stage(t + step);
      cp_async_wait_but_one();
      __syncwarp();
    }
    Cols c_[V], o_[V], f_[V], d[V], g_[V];
    if (kHeld) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        c_[v] = rn[v].get(), o_[v] = ro[v].get(), f_[v] = rb[v].get(), d[v] = rd[v].get();
        if (FULL) g_[v] = rg[v].get();
      }
      fetch(t + step);
    }
    auto c = [&](int v) { return kHeld ? c_[v] : half(v); };
    auto o = [&](int v) { return kHeld ? o_[v] : wide(V + v); };
    auto f = [&](int v) { return kHeld ? f_[v] : half(V + v); };
    auto g = [&](int v) { return kHeld ? g_[v] : half(2 * V + v); };
    auto d0 = [&](int v) { return kHeld ? d[v] : a.dout ? wide(v) : Cols::of(0.0f); };
    float s[2];
    if (a.dn) {
      s[0] = s[1] = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (on[v]) {
          s[0] += dot8(o(v), o(v));
          s[1] += dot8(next[v], c(v) * o(v));
        }
      sums(s, me);
      const float r = inv_rms(s[0], inv_k, a.eps), q = s[1] * r * inv_k * r;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (on[v] && t < a.T) sn[v] = fma8(c(v) * o(v), r, sn[v]);
        d[v] = fma8(fma8(o(v), -q, c(v) * next[v]), r, d0(v));
      }
    } else if (!kHeld) {
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = d0(v);
    }
    if (a.dx) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (on[v] && t < a.T) put8(static_cast<S*>(a.dx) + row + col[v], d[v] * a.alpha);
    }
    if (a.b) {
      float r = 1.0f, q = 0.0f;
      if (a.w_post) {
        s[0] = s[1] = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (on[v]) {
            s[0] += dot8(f(v), f(v));
            s[1] += dot8(FULL ? post[v] * g(v) : post[v], d[v] * f(v));
          }
        sums(s, me);
        r = inv_rms(s[0], inv_k, a.eps);
        q = s[1] * r * inv_k * r;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!on[v] || t >= a.T) continue;
        Cols e = d[v] * post[v], df = d[v] * f(v);
        if (FULL) {
          put8(a.dgate_full + row + col[v], df * r * post[v]);
          df = df * g(v);
          e = e * g(v);
        }
        sb[v] = fma8(df, r, sb[v]);
        // (without its norm b is no part of its gradient, and 0 times an infinity would be)
        put8(a.db + row + col[v], a.w_post ? fma8(f(v), -q, e) * r : e);
      }
    }
  }
  if constexpr (ONE) {
    __shared__ __align__(16) float cols[2][8 * NT];
    put8(&cols[0][8 * threadIdx.x], sb[0]);
    put8(&cols[1][8 * threadIdx.x], sn[0]);
    __syncwarp();
    cluster_sync_all();
    for (int c = static_cast<int>(blockIdx.x) * NT + threadIdx.x; c < a.K; c += kOneCtas * NT) {
      float post = 0.0f, next = 0.0f;
      for (int cta = 0; cta < kOneCtas; ++cta)
        for (int team = 0; team < me.rows; ++team) {
          const uint32_t at = mapa_shared(smem_u32(&cols[0][8 * a.row_threads * team + c]), cta);
          float p, n;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p) : "r"(at));
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(n) : "r"(at + static_cast<uint32_t>(sizeof(cols[0]))));
          post += p;
          next += n;
        }
      put_columns(a, c, post, next);
    }
    __syncwarp();
    cluster_sync_all();  // none of the CTAs leaves before its sums have been read
    return;
  }
  if constexpr (NT == 256) {
    if (me.rows > 1) {  // the CTA's rows, joined in their order
      __shared__ __align__(16) float cols[2][8 * NT];
      put8(&cols[0][8 * threadIdx.x], sb[0]);
      put8(&cols[1][8 * threadIdx.x], sn[0]);
      __syncthreads();
      for (int c = threadIdx.x; c < a.K; c += NT) {
        float post = 0.0f, next = 0.0f;
        for (int team = 0; team < me.rows; ++team) {
          post += cols[0][8 * a.row_threads * team + c];
          next += cols[1][8 * a.row_threads * team + c];
        }
        float* p = a.parts + static_cast<long long>(blockIdx.x) * 2 * a.K + c;
        p[0] = post;
        p[a.K] = next;
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!on[v]) continue;
    float* p = a.parts + static_cast<long long>(blockIdx.x) * 2 * a.K + col[v];
    if (a.dw_post || a.dgate_col) put8(p, sb[v]);
    if (a.dw_next) put8(p + a.K, sn[v]);
  }
}

// Sums the parts in their order and gives the parameters' gradients: 8 columns a CTA,
// 32 threads a column with every 32nd part each, a warp a column for what they have.
__global__ void __launch_bounds__(256) norm_join_reduce_kernel(const float* __restrict__ parts, int P, int K,
                                                               float beta, const float* w_post, const float* gate,
                                                               float* dw_post, float* dgate, float* dw_next) {
  __shared__ float sums[32][9];
  griddep_launch_dependents();
  griddep_wait();
  const bool next = blockIdx.y == 1;
  if (next ? !dw_next : !dw_post && !dgate) return;
  const int c = threadIdx.x & 7, group = threadIdx.x >> 3;
  const float* p = parts + static_cast<long long>(blockIdx.y) * K + blockIdx.x * 8 + c;
  float s = 0.0f;
  for (int i = group; i < P; i += 32 * 10) {
    float v[10];  // all on their way at once: up to 320 parts in one round
#pragma unroll
    for (int j = 0; j < 10; ++j) v[j] = i + 32 * j < P ? p[static_cast<long long>(i + 32 * j) * 2 * K] : 0.0f;
#pragma unroll
    for (int j = 0; j < 10; ++j) s += v[j];
  }
  sums[group][c] = s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 8 + warp;
  float g = 1.0f, w = 1.0f;
  if (!next && dw_post && gate) g = gate[col];
  if (!next && dgate && w_post) w = w_post[col];
  __syncthreads();
  const float total = warp_sum(sums[lane][warp]);
  if (lane != 0) return;
  if (next) {
    dw_next[col] = total;
  } else {
    if (dw_post) dw_post[col] = beta * total * g;
    if (dgate) dgate[col] = beta * total * w;
  }
}

// How T rows of K columns are laid out: `vectors` of 8 columns a thread, 512 threads an
// SM (128 registers each).
struct Shape {
  int row_threads, threads, teams, grid;
  Shape(int64_t T, int64_t K, int vectors, int sms) {
    const int64_t each = 8 * 32 * vectors;  // columns of a warp
    row_threads = static_cast<int>((K + each - 1) / each * 32);
    threads = row_threads <= 256 ? 256 : 512;
    teams = threads / row_threads;
    const long long need = (T + teams - 1) / teams, room = static_cast<long long>(sms) * (512 / threads);
    grid = static_cast<int>(need < room ? need : room);
  }
};

// Vectors a thread.  The backward pass holds more for each: two only where one would
// take over 512 threads.
constexpr int kForward = 2;
int backward_vectors(int64_t K) { return K > 8 * 512 ? 2 : 1; }
// Rows that the backward pass gives one cluster: up to eight a CTA (and row of a CTA).
bool one_cluster(int64_t T, int64_t K) {
  const int row_threads = static_cast<int>((K / 8 + 31) / 32 * 32);
  return T > 0 && row_threads <= 512 && T <= 8 * kOneCtas * (row_threads <= 256 ? 256 / row_threads : 1);
}

template <typename S, bool FULL>
cudaError_t forward(const NormJoinArgs& a, const Shape& sh, cudaStream_t stream) {
  const bool over = launch_over(8 * a.T * a.K, stream);
  return sh.threads == 256
             ? launch_short(over, norm_join_kernel<S, kForward, 256, FULL>, dim3(sh.grid), dim3(256), 0, stream, a)
             : launch_short(over, norm_join_kernel<S, kForward, 512, FULL>, dim3(sh.grid), dim3(512), 0, stream, a);
}
template <typename S, bool FULL>
cudaError_t backward(const NormJoinBwdArgs& a, const Shape& sh, bool over, cudaStream_t stream) {
  if (one_cluster(a.T, a.K)) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kOneCtas);
    cfg.blockDim = dim3(sh.threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kOneCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return sh.threads == 256 ? cudaLaunchKernelEx(&cfg, norm_join_bwd_kernel<S, 1, 256, FULL, true>, a)
                             : cudaLaunchKernelEx(&cfg, norm_join_bwd_kernel<S, 1, 512, FULL, true>, a);
  }
  if (backward_vectors(a.K) == 2) {
    constexpr int kSmem = 2 * 2 * static_cast<int>(sizeof(S) + 2 + FULL) * 16 * 512;  // two rows
    static std::atomic<uint64_t> done{0};
    const auto kernel = norm_join_bwd_kernel<S, 2, 512, FULL, false>;
    const cudaError_t e = allow_smem(kernel, kSmem, done);
    if (e != cudaSuccess) return e;
    return launch_short(over, kernel, dim3(sh.grid), dim3(512), kSmem, stream, a);
  }
  return sh.threads == 256
             ? launch_short(over, norm_join_bwd_kernel<S, 1, 256, FULL, false>, dim3(sh.grid), dim3(256), 0, stream, a)
             : launch_short(over, norm_join_bwd_kernel<S, 1, 512, FULL, false>, dim3(sh.grid), dim3(512), 0, stream, a);
}

}  // namespace

int norm_join_parts(int64_t T, int64_t K, int sms) {
  if (one_cluster(T, K)) return 0;
  const Shape sh(T, K, backward_vectors(K), sms);
  return sh.grid;
}

cudaError_t launch_norm_join(const NormJoinArgs& args, int sms, cudaStream_t stream) {
  NormJoinArgs a = args;
  const Shape sh(a.T, a.K, kForward, sms);
  a.row_threads = sh.row_threads;
  if (a.gate_full) return a.f32 ? forward<float, true>(a, sh, stream) : forward<uint16_t, true>(a, sh, stream);
  return a.f32 ? forward<float, false>(a, sh, stream) : forward<uint16_t, false>(a, sh, stream);
}

cudaError_t launch_norm_join_bwd(const NormJoinBwdArgs& args, int sms, cudaStream_t stream) {
  NormJoinBwdArgs a = args;
  const Shape sh(a.T, a.K, backward_vectors(a.K), sms);
  a.row_threads = sh.row_threads;
  const bool over = launch_over(12 * a.T * a.K, stream);
  cudaError_t e = cudaSuccess;
  if (a.T > 0) {
    if (a.gate_full)
      e = a.f32 ? backward<float, true>(a, sh, over, stream) : backward<uint16_t, true>(a, sh, over, stream);
    else
      e = a.f32 ? backward<float, false>(a, sh, over, stream) : backward<uint16_t, false>(a, sh, over, stream);
  }
  if (e != cudaSuccess || one_cluster(a.T, a.K) || !(a.dw_post || a.dgate_col || a.dw_next)) return e;
  return launch_short(over, norm_join_reduce_kernel, dim3(static_cast<unsigned>(a.K / 8), 2), dim3(256), 0, stream,
                      static_cast<const float*>(a.parts), sh.grid, static_cast<int>(a.K), a.beta, a.w_post,
                      a.gate_col, a.dw_post, a.dgate_col, a.dw_next);
}

}  // namespace gmm
