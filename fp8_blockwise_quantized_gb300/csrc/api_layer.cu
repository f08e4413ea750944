// Host side of the entry points around the experts (include/gmm.h): the router,
// the sorted rows, the norms with their residual stream, and gradient clipping.
// Nothing here allocates device memory or synchronizes.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <utility>
#include <vector>

#include "gmm.h"
#include "common.cuh"
#include "host.cuh"
#include "kernels.cuh"

using namespace gmm;

namespace {

template <typename... P>
bool all_aligned(P... p) {
  return (((reinterpret_cast<uintptr_t>(p) & 15u) == 0) && ...);
}

gmm_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? GMM_OK : host_cuda_fail(e, what); }

constexpr int kMaxChoices = 32;
constexpr int64_t kMaxColumns = 1 << 24;
constexpr int64_t kMaxNormColumns = 8192;  // 1024 threads of 8

gmm_status check_choices(int64_t T, int k) {
  return T < 0 || k < 1 || k > kMaxChoices || T > INT32_MAX / k ? GMM_ERR_SHAPE : GMM_OK;
}
gmm_status check_columns(int64_t K, int unit) {
  return K < unit || K % unit != 0 || K > kMaxColumns ? GMM_ERR_SHAPE : GMM_OK;
}

gmm_status check_route(gmm_type type, int64_t T, int E, int k, gmm_score score) {
  if (check_choices(T, k) != GMM_OK || E < 1 || E > kMaxGroups || k > E) return GMM_ERR_SHAPE;
  if ((type != GMM_BF16 && type != GMM_F32) || (score != GMM_SOFTMAX && score != GMM_SIGMOID))
    return GMM_ERR_UNSUPPORTED;
  return GMM_OK;
}

RouteArgs route_args(const void* logits, gmm_type type, int64_t T, int E, int k, gmm_score score, int renorm,
                     float scale) {
  RouteArgs a{};
  a.logits = logits;
  a.T = T;
  a.E = E;
  a.k = k;
  a.f32 = type == GMM_F32;
  a.softmax = score == GMM_SOFTMAX;
  a.renorm = renorm != 0;
  a.scale = scale;
  return a;
}

// What the calls on rows share: sizes, pointers, the device.
gmm_status check_rows(int64_t T, int k, int64_t K, int unit, bool pointers, bool aligned, int* sms) {
  gmm_status st = check_choices(T, k);
  if (st != GMM_OK || (st = check_columns(K, unit)) != GMM_OK) return st;
  if (T > 0 && !pointers) return GMM_ERR_NULL;
  if (!aligned) return GMM_ERR_ALIGN;
  return T > 0 ? host_device_sms(sms) : GMM_OK;
}

gmm_status check_join(int64_t T, int64_t K, gmm_type type, const void* b, const void* w_post, const void* gate,
                      float eps) {
  if (T < 0 || T > INT32_MAX || check_columns(K, 8) != GMM_OK || K > kMaxNormColumns) return GMM_ERR_SHAPE;
  if ((type != GMM_BF16 && type != GMM_F32) || !(eps >= 0.0f)) return GMM_ERR_UNSUPPORTED;
  return T > 0 && !b && (w_post || gate) ? GMM_ERR_NULL : GMM_OK;  // without tokens b has no address
}

// Whether an output shares memory with another one, or with a gradient that is not its
// own: the CTAs would scale it twice, or read it scaled.
bool outputs_overlap(const std::vector<ClipTensor>& t) {
  using Range = std::pair<uintptr_t, uintptr_t>;
  const auto range = [](const ClipTensor& c, const void* p) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return Range(at, at + static_cast<uintptr_t>(c.count) * (c.f32 ? 4 : 2));
  };
  std::vector<Range> out;
  out.reserve(t.size());
  bool elsewhere = false;
  for (const ClipTensor& c : t) {
    out.push_back(range(c, c.dst));
    elsewhere |= c.dst != c.src;
  }
  std::sort(out.begin(), out.end());
  for (size_t i = 1; i < out.size(); ++i)
    if (out[i].first < out[i - 1].second) return true;
  if (!elsewhere) return false;
  for (const ClipTensor& c : t) {
    const Range in = range(c, c.src), own = range(c, c.dst);
    // the first output that ends behind the gradient's start (they are disjoint, so sorted by their ends too)
    auto it = std::upper_bound(out.begin(), out.end(), in.first,
                               [](uintptr_t at, const Range& r) { return at < r.second; });
    for (; it != out.end() && it->first < in.second; ++it)
      if (!(*it == own && own == in)) return true;
  }
  return false;
}

}  // namespace

extern "C" {

gmm_status gmm_route(const void* logits, gmm_type logits_type, const float* bias, int64_t T, int E, int k,
                     gmm_score score, int renorm, float scale, int32_t* ids, float* weights, void* stream) {
  gmm_status st = check_route(logits_type, T, E, k, score);
  if (st != GMM_OK) return st;
  if (T > 0 && (!logits || !ids || !weights)) return GMM_ERR_NULL;
  if (!all_aligned(logits, bias, ids, weights)) return GMM_ERR_ALIGN;
  if (T == 0) return GMM_OK;
  int sms = 0;
  if ((st = host_device_sms(&sms)) != GMM_OK) return st;
  RouteArgs a = route_args(logits, logits_type, T, E, k, score, renorm, scale);
  a.bias = bias;
  a.ids_out = ids;
  a.weights = weights;
  return launched(launch_route(a, static_cast<cudaStream_t>(stream)), "route_kernel launch");
}

gmm_status gmm_route_bwd(const float* dweights, const void* logits, gmm_type logits_type, const int32_t* ids, int64_t T,
                         int E, int k, gmm_score score, int renorm, float scale, void* dlogits, void* stream) {
  gmm_status st = check_route(logits_type, T, E, k, score);
  if (st != GMM_OK) return st;
  if (T > 0 && (!dweights || !logits || !ids || !dlogits)) return GMM_ERR_NULL;
  if (!all_aligned(dweights, logits, ids, dlogits)) return GMM_ERR_ALIGN;
  if (T == 0) return GMM_OK;
  int sms = 0;
  if ((st = host_device_sms(&sms)) != GMM_OK) return st;
  RouteArgs a = route_args(logits, logits_type, T, E, k, score, renorm, scale);
  a.dweights = dweights;
  a.ids = ids;
  a.dlogits = dlogits;
  return launched(launch_route_bwd(a, static_cast<cudaStream_t>(stream)), "route_bwd_kernel launch");
}

size_t gmm_sort_rows_scratch_bytes(int64_t N, int G) {
  return N < 0 || N > INT32_MAX || G < 1 || G > kMaxGroups ? 0 : sort_scratch_bytes(N, G);
}

gmm_status gmm_sort_rows(const int32_t* ids, int64_t N, int G, int32_t* rows, int32_t* group_sizes, void* scratch,
                         size_t scratch_bytes, void* stream) {
  if (N < 0 || N > INT32_MAX || G < 1 || G > kMaxGroups) return GMM_ERR_SHAPE;
  if (!group_sizes || (N > 0 && (!ids || !rows))) return GMM_ERR_NULL;
  if (!all_aligned(ids, rows, group_sizes, scratch)) return GMM_ERR_ALIGN;
  const size_t need = sort_scratch_bytes(N, G);
  if (need && (!scratch || scratch_bytes < need)) return GMM_ERR_WORKSPACE;
  int sms = 0;
  const gmm_status st = host_device_sms(&sms);
  if (st != GMM_OK) return st;
  return launched(launch_sort_rows(ids, N, G, rows, group_sizes, scratch, static_cast<cudaStream_t>(stream)),
                  "sort_rows launch");
}

gmm_status gmm_gather_rows(const void* x, const int32_t* rows, int64_t T, int k, int64_t K, void* out, void* stream) {
  int sms = 0;
  const gmm_status st = check_rows(T, k, K, 8, x && rows && out, all_aligned(x, rows, out), &sms);
  if (st != GMM_OK || T == 0) return st;
  return launched(launch_gather_rows(x, rows, T, k, K, out, static_cast<cudaStream_t>(stream)), "gather_kernel launch");
}

gmm_status gmm_gather_quantize(const void* x, const int32_t* rows, int64_t T, int k, int64_t K, void* xq, float* xs,
                               void* stream) {
  int sms = 0;
  const gmm_status st = check_rows(T, k, K, 128, x && rows && xq && xs, all_aligned(x, rows, xq, xs), &sms);
  if (st != GMM_OK || T == 0) return st;
  return launched(launch_gather_quantize(x, rows, T, k, K, xq, xs, static_cast<cudaStream_t>(stream)),
                  "gather_quantize_kernel launch");
}

gmm_status gmm_gather_mx4_quantize(const void* x, const int32_t* rows, int64_t T, int k, int64_t K, void* xq, void* xs,
                                   void* stream) {
  int sms = 0;
  const gmm_status st = check_rows(T, k, K, 128, x && rows && xq && xs, all_aligned(x, rows, xq, xs), &sms);
  if (st != GMM_OK || T == 0) return st;
  return launched(launch_gather_mx4(x, rows, T, k, K, xq, xs, static_cast<cudaStream_t>(stream)),
                  "gather_mx4_kernel launch");
}

gmm_status gmm_combine_rows(const void* y, const int32_t* rows, const float* weights, int64_t T, int k, int64_t K,
                            void* out, void* stream) {
  int sms = 0;
  const gmm_status st = check_rows(T, k, K, 8, y && rows && out, all_aligned(y, rows, weights, out), &sms);
  if (st != GMM_OK || T == 0) return st;
  return launched(launch_combine_rows(y, rows, weights, T, k, K, out, static_cast<cudaStream_t>(stream)),
                  "combine_kernel launch");
}

gmm_status gmm_combine_rows_bwd(const void* dout, const void* y, const int32_t* rows, const float* weights, int64_t T,
                                int k, int64_t K, void* dy, float* dweights, void* stream) {
  int sms = 0;
  const gmm_status st = check_rows(T, k, K, 8, dout && y && rows && weights && dy && dweights,
                                   all_aligned(dout, y, rows, weights, dy, dweights), &sms);
  if (st != GMM_OK || T == 0) return st;
  return launched(launch_combine_rows_bwd(dout, y, rows, weights, T, k, K, dy, dweights, sms,
                                          static_cast<cudaStream_t>(stream)),
                  "combine_bwd_kernel launch");
}

gmm_status gmm_norm_join(const void* x, gmm_type stream_type, const void* b, const float* w_post, const void* gate,
                         int gate_rows, const float* w_next, int64_t T, int64_t K, float residual_scale,
                         float block_scale, float eps, void* out, void* n, void* stream) {
  gmm_status st = check_join(T, K, stream_type, b, w_post, gate, eps);
  if (st != GMM_OK) return st;
  if (T > 0 && (!x || (b && !out) || (w_next && !n) || (!b && !w_next))) return GMM_ERR_NULL;
  if (!all_aligned(x, b, w_post, gate, w_next, out, n)) return GMM_ERR_ALIGN;
  if (T == 0) return GMM_OK;
  int sms = 0;
  if ((st = host_device_sms(&sms)) != GMM_OK) return st;
  NormJoinArgs a{};
  a.x = x;
  a.b = static_cast<const uint16_t*>(b);
  a.w_post = w_post;
  a.gate_col = gate_rows ? nullptr : static_cast<const float*>(gate);
  a.gate_full = gate_rows ? static_cast<const uint16_t*>(gate) : nullptr;
  a.w_next = w_next;
  a.out = out;
  a.n = static_cast<uint16_t*>(n);
  a.T = T;
  a.K = static_cast<int>(K);
  a.f32 = stream_type == GMM_F32;
  a.alpha = b ? residual_scale : 1.0f;
  a.beta = block_scale;
  a.eps = eps;
  return launched(launch_norm_join(a, sms, static_cast<cudaStream_t>(stream)), "norm_join_kernel launch");
}

size_t gmm_norm_join_bwd_scratch_bytes(int64_t T, int64_t K) {
  int sms = 0;
  if (T < 0 || T > INT32_MAX || check_columns(K, 8) != GMM_OK || K > kMaxNormColumns ||
      host_device_sms(&sms) != GMM_OK)
    return 0;
  return static_cast<size_t>(norm_join_parts(T, K, sms)) * 2 * K * sizeof(float);
}

gmm_status gmm_norm_join_bwd(const void* dout, const void* dn, const void* out, gmm_type stream_type, const void* b,
                             const float* w_post, const void* gate, int gate_rows, const float* w_next, int64_t T,
                             int64_t K, float residual_scale, float block_scale, float eps, void* dx, void* db,
                             float* dw_post, void* dgate, float* dw_next, void* scratch, size_t scratch_bytes,
                             void* stream) {
  gmm_status st = check_join(T, K, stream_type, b, w_post, gate, eps);
  if (st != GMM_OK) return st;
  if ((dw_post && !w_post) || (dgate && !gate) || (dw_next && !w_next)) return GMM_ERR_NULL;
  if (T > 0 && ((dn && (!w_next || !out)) || (b && !db) || (gate && gate_rows && !dgate))) return GMM_ERR_NULL;
  if (!all_aligned(dout, dn, out, b, w_post, gate, w_next, dx, db, dw_post, dgate, dw_next, scratch))
    return GMM_ERR_ALIGN;
  int sms = 0;
  if ((st = host_device_sms(&sms)) != GMM_OK) return st;
  const size_t need = static_cast<size_t>(norm_join_parts(T, K, sms)) * 2 * K * sizeof(float);
  if (need && (!scratch || scratch_bytes < need)) return GMM_ERR_WORKSPACE;
  NormJoinBwdArgs a{};
  a.dout = dout;
  a.dn = static_cast<const uint16_t*>(dn);
  a.out = out;
  a.b = static_cast<const uint16_t*>(b);
  a.w_post = w_post;
  a.gate_col = gate_rows ? nullptr : static_cast<const float*>(gate);
  a.gate_full = gate_rows ? static_cast<const uint16_t*>(gate) : nullptr;
  a.w_next = w_next;
  a.dx = dx;
  a.db = static_cast<uint16_t*>(db);
  a.dw_post = dw_post;
  a.dgate_col = gate_rows ? nullptr : static_cast<float*>(dgate);
  a.dgate_full = gate_rows ? static_cast<uint16_t*>(dgate) : nullptr;
  a.dw_next = dw_next;
  a.parts = static_cast<float*>(scratch);
  a.T = T;
  a.K = static_cast<int>(K);
  a.f32 = stream_type == GMM_F32;
  a.alpha = b ? residual_scale : 1.0f;
  a.beta = block_scale;
  a.eps = eps;
  return launched(launch_norm_join_bwd(a, sms, static_cast<cudaStream_t>(stream)), "norm_join_bwd launch");
}

size_t gmm_clip_grads_scratch_bytes(int n, int64_t total) {
  int sms = 0;
  return n < 0 || total < 0 || host_device_sms(&sms) != GMM_OK ? 0 : clip_scratch_bytes(n, total, sms);
}

gmm_status gmm_clip_grads(const void* const* grads, void* const* out, const int64_t* counts, const int32_t* types,
                          int n, float max_norm, float* norm, void* scratch, size_t scratch_bytes, void* stream) {
  if (n < 0) return GMM_ERR_SHAPE;
  if (!(max_norm >= 0.0f)) return GMM_ERR_UNSUPPORTED;
  if (!norm || (n > 0 && (!grads || !counts || !types))) return GMM_ERR_NULL;
  constexpr int64_t kMost = 1LL << 42;  // elements, so that the chunks' numbers are 32 bits
  int64_t total = 0;
  for (int i = 0; i < n; ++i) {
    if (types[i] != GMM_BF16 && types[i] != GMM_F32) return GMM_ERR_UNSUPPORTED;
    if (counts[i] < 0 || counts[i] > kMost || (total += counts[i]) > kMost) return GMM_ERR_SHAPE;
    if (counts[i] == 0) continue;
    if (!grads[i] || (out && !out[i])) return GMM_ERR_NULL;
    const uintptr_t at = reinterpret_cast<uintptr_t>(grads[i]) | (out ? reinterpret_cast<uintptr_t>(out[i]) : 0);
    if (at & (types[i] == GMM_F32 ? 3u : 1u)) return GMM_ERR_ALIGN;
  }
  if (!all_aligned(norm, scratch)) return GMM_ERR_ALIGN;
  try {
    std::vector<ClipTensor> t;
    t.reserve(n);
    for (int i = 0; i < n; ++i)
      if (counts[i] > 0)
        t.push_back({grads[i], out ? out[i] : const_cast<void*>(grads[i]), counts[i], types[i] == GMM_F32});
    if (outputs_overlap(t)) return host_fail(GMM_ERR_UNSUPPORTED, "clip_grads: outputs overlap");
    int sms = 0;
    const gmm_status st = host_device_sms(&sms);
    if (st != GMM_OK) return st;
    const size_t need = clip_scratch_bytes(n, total, sms);
    if (need && (!scratch || scratch_bytes < need)) return GMM_ERR_WORKSPACE;
    return launched(launch_clip(t.data(), static_cast<int>(t.size()), max_norm, out == nullptr,
                                scratch, norm, sms, static_cast<cudaStream_t>(stream)),
                    "clip_grads launch");
  } catch (...) {
    return host_fail(GMM_ERR_CUDA, "out of host memory");
  }
}

}  // extern "C"
