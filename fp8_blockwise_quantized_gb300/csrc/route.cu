// The router: the k experts of each token and their weights, and the gradient
// of the logits.
//
// A warp takes a token and holds its E logits in registers, expert i * 32 + lane
// in lane's word i, so that every load and store of a word is contiguous.  Bound by
// its instructions (60 % of the issue slots, backward 66 %) and the wait for a token's
// logits together, and for few tokens by the chain of the choice.  Forward, 8192
// tokens, 256 experts, 8 choices: 7.6 us (k rounds of a warp-wide maximum, each lane
// looking through its words: 11.6; each keeping its two best: 9.7); backward 6.7.
//
// The choice: the k-th largest of the lanes' best keys is at most the k-th largest key,
// so the experts that reach it (a few more than k) are all that can be chosen.  They
// are gathered in the order of their ids, one a lane, and each counts those before it.
// Where more than 32 reach it (many equal keys, or few lanes with any) the choices are
// made one after the other.
#include "common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace gmm {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ float minus_inf() { return __int_as_float(0xff800000); }
// A logit in fp32; NaN stands for an expert that is not there.
__device__ __forceinline__ float logit_of(const float* p) { return fmaxf(__ldg(p), minus_inf()); }
__device__ __forceinline__ float logit_of(const uint16_t* p) {
  return fmaxf(__uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16), minus_inf());
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) {
  *p = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xffffu);
}

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// The score that renorm divides by the chosen ones' sum, as its logarithm: the
// logit itself (softmax), or log sigmoid(v), which keeps its value where the
// sigmoid is below the smallest float.
__device__ __forceinline__ float log_score(float v, bool softmax) {
  return softmax ? v : fminf(v, 0.0f) - log1pf(expf(-fabsf(v)));
}

// exp(v - the warp's largest) over its sum: 0 at -inf, and everywhere when all are -inf.
__device__ __forceinline__ float share_of(float v) {
  const float top = warp_max(v);
  const float e = v > minus_inf() ? expf(v - top) : 0.0f;
  const float sum = warp_sum(e);
  return e > 0.0f || e != e ? e / sum : 0.0f;
}

// Largest logit of the row and the sum of exp(logit - largest).
template <int V>
__device__ __forceinline__ void row_sum(const float (&l)[V], float* top, float* sum) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
  m = warp_max(m);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) s += l[i] > minus_inf() ? expf(l[i] - m) : 0.0f;
  *top = m;
  *sum = warp_sum(s);
}

__device__ __forceinline__ float warp_most(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

constexpr int kWarps = 4;

template <typename L, int V>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const L* __restrict__ logits,
                                                            const float* __restrict__ bias, long long T, int E, int k,
                                                            int softmax, int renorm, float scale,
                                                            int32_t* __restrict__ ids, float* __restrict__ weights) {
  griddep_launch_dependents();
  griddep_wait();  // the logits may come from the previous kernel
  __shared__ float keys[kWarps][32];
  __shared__ int names[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (t >= T) return;
  const L* row = logits + t * E;
  float key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = 32 * i + lane < E ? logit_of(row + 32 * i + lane) : minus_inf();
  float top = 0.0f, sum = 1.0f;
  if (softmax && !renorm) row_sum<V>(key, &top, &sum);
  if (bias) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (32 * i + lane < E) key[i] = fmaxf(key[i] + __ldg(bias + 32 * i + lane), minus_inf());
  }
  float best = key[0];
#pragma unroll
  for (int i = 1; i < V; ++i) best = fmaxf(best, key[i]);
  float least = minus_inf();  // what a chosen key reaches; it is above -inf too
  for (int j = 0; j < k; ++j) {
    least = warp_most(best);
    if (best == least) best = minus_inf();
  }
  int found = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool in = key[i] >= least && key[i] > minus_inf();
    const uint32_t with = __ballot_sync(kAll, in);
    const int at = found + __popc(with & ((1u << lane) - 1u));
    if (in && at < 32) keys[warp][at] = key[i], names[warp][at] = 32 * i + lane;
    found += __popc(with);
  }
  __syncwarp();
  int mine = -1, place = k;  // this lane's expert and which choice it is
  if (found <= 32) {
    if (lane < found) {
      const float own = keys[warp][lane];
      mine = names[warp][lane];
      place = 0;
      for (int j = 0; j < found; ++j) {
        const float other = keys[warp][j];
        place += other > own || (other == own && j < lane);
      }
    }
    // the empty choices' lanes
    if (lane >= found) place = lane;
  } else {
    place = lane;
    for (int j = 0; j < k; ++j) {
      float first = key[0];
      int at = 0;
#pragma unroll
      for (int i = 1; i < V; ++i)
        if (key[i] > first) first = key[i], at = i;
      const float most = warp_most(first);
      if (!(most > minus_inf())) break;
      const uint32_t id = __reduce_min_sync(kAll, first == most ? 32u * at + lane : ~0u);
      if (lane == j) mine = static_cast<int>(id);
      const int gone = lane == (id & 31u) ? static_cast<int>(id >> 5) : -1;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == gone) key[i] = minus_inf();
    }
  }
  if (place >= k) mine = -1;
  const float v = mine >= 0 ? logit_of(row + mine) : minus_inf();
  float w;
  if (renorm)
    w = share_of(mine >= 0 ? log_score(v, softmax) : minus_inf());
  else
    w = mine < 0 ? 0.0f : softmax ? expf(v - top) / sum : sigmoid(v);
  if (place < k) {
    ids[t * k + place] = mine;
    weights[t * k + place] = scale * w;
  }
}

template <typename L, int V>
__global__ void __launch_bounds__(32 * kWarps) route_bwd_kernel(const float* __restrict__ dweights,
                                                                const L* __restrict__ logits,
                                                                const int32_t* __restrict__ ids, long long T, int E,
                                                                int k, int softmax, int renorm, float scale,
                                                                L* __restrict__ dlogits) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  const L* row = logits + t * E;
  int id = lane < k ? __ldg(ids + t * k + lane) : -1;
  if (id >= E) id = -1;
  const float g = id >= 0 ? scale * __ldg(dweights + t * k + lane) : 0.0f;
  const float v = id >= 0 ? logit_of(row + id) : minus_inf();
  const bool whole = softmax && !renorm;  // every expert's logit counts
  float p[V], total = 0.0f, mine = 0.0f;
  float d;  // what choice `lane` adds to its expert
  if (whole) {
    float top, sum;
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = 32 * i + lane < E ? logit_of(row + 32 * i + lane) : minus_inf();
    row_sum<V>(p, &top, &sum);
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = p[i] > minus_inf() ? expf(p[i] - top) * inv : 0.0f;
    if (id >= 0 && v > minus_inf()) mine = expf(v - top) * inv;
    total = warp_sum(g * mine);
    d = g * mine;
  } else if (renorm) {
    const float q = share_of(id >= 0 ? log_score(v, softmax) : minus_inf());
    d = q * (g - warp_sum(g * q));
    if (!softmax) d *= sigmoid(-v);
  } else {
    const float e = expf(-fabsf(v));
    d = g * (e / ((1.0f + e) * (1.0f + e)));
  }
  // an expert that a token names twice gets both, in the order of the choices
  bool twice = false;
  float rest = d;
  for (int j = 0; j < k; ++j) {
    const int to = __shfl_sync(kAll, id, j);
    const float add = __shfl_sync(kAll, d, j);
    if (id >= 0 && id == to && lane != j) {
      twice |= lane > j;  // the first of them writes the sum
      if (lane < j) rest += add;
    }
  }
  if (whole) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (32 * i + lane < E) put(dlogits + t * E + 32 * i + lane, -p[i] * total);
    rest -= mine * total;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (32 * i + lane < E) put(dlogits + t * E + 32 * i + lane, 0.0f);
  }
  __syncwarp();  // the row is written before the choices' words in it
  if (id >= 0 && !twice) put(dlogits + t * E + id, rest);
}

template <typename F>
cudaError_t by_words(int E, F&& launch) {
  if (E <= 32) return launch(std::integral_constant<int, 1>());
  if (E <= 64) return launch(std::integral_constant<int, 2>());
  if (E <= 128) return launch(std::integral_constant<int, 4>());
  if (E <= 256) return launch(std::integral_constant<int, 8>());
  if (E <= 512) return launch(std::integral_constant<int, 16>());
  if (E <= 1024) return launch(std::integral_constant<int, 32>());
  if (E <= 2048) return launch(std::integral_constant<int, 64>());
  return launch(std::integral_constant<int, 128>());
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.T + kWarps - 1) / kWarps)), block(32 * kWarps);
  // (a fifth of the memory's rate)
  const bool over = launch_over(5 * a.T * a.E * (a.f32 ? 4 : 2), stream);
  return by_words(a.E, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (a.f32)
      return launch_short(over, route_kernel<float, V>, grid, block, 0, stream, static_cast<const float*>(a.logits),
                          a.bias, a.T, a.E, a.k, a.softmax, a.renorm, a.scale, a.ids_out, a.weights);
    return launch_short(over, route_kernel<uint16_t, V>, grid, block, 0, stream, static_cast<const uint16_t*>(a.logits),
                        a.bias, a.T, a.E, a.k, a.softmax, a.renorm, a.scale, a.ids_out, a.weights);
  });
}

cudaError_t launch_route_bwd(const RouteArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.T + kWarps - 1) / kWarps)), block(32 * kWarps);
  // (a fifth of the memory's rate)
  const bool over = launch_over(5 * a.T * a.E * (a.f32 ? 4 : 2), stream);
  return by_words(a.E, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (a.f32)
      return launch_short(over, route_bwd_kernel<float, V>, grid, block, 0, stream, a.dweights,
                          static_cast<const float*>(a.logits), a.ids, a.T, a.E, a.k, a.softmax, a.renorm, a.scale,
                          static_cast<float*>(a.dlogits));
    return launch_short(over, route_bwd_kernel<uint16_t, V>, grid, block, 0, stream, a.dweights,
                        static_cast<const uint16_t*>(a.logits), a.ids, a.T, a.E, a.k, a.softmax, a.renorm, a.scale,
                        static_cast<uint16_t*>(a.dlogits));
  });
}

}  // namespace gmm
