// The global norm of many gradients, and their scaling to a largest norm.
//
// The tensors come as a table in the launch's parameters, cut into chunks of one
// length; a CTA finds a chunk's tensor by bisection.  The first pass leaves a sum of
// squares a CTA; each CTA of the second adds them all up in their order, so that the
// norm is one number whatever the schedule, and scales.  The second pass takes the
// chunks backwards, from those that may still be in the L2 (60 M values 83.7 us, forwards
// 85.6; no difference at 805 M, 725 us, where two reads and a write take 724).
//
// Sums are pairs of fp32 values, a sum and what its roundings left (a thread's share of
// one chunk, up to 128 squares, is one value), and the norm and the factor come from both,
// so that each is rounded once.  That holds while every square keeps its bits in fp32; a
// CTA that meets a sum outside that range adds its values up in double, of which this GPU
// does two a cycle and SM (sums in double throughout: 19.7 us for 60 tensors of 3 M values,
// for 8.5).  So are the products where the factor, max_norm / norm, is not a normal number
// (60 M values: 383 us for 57).
//
// A few values are one launch's: a cluster's CTAs, which read each other's sums and
// keep their chunks' values in the caches.  It saves the host a launch and the caller
// the scratch.
#include "common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace gmm {

namespace {

// A chunk is 256 threads' at a time: a CTA's, or in the one launch for a few values a
// quarter of a CTA's.
constexpr int kThreads = 256, kOneThreads = 1024, kOneCtas = 8;

template <int N>
struct ClipTable {
  const void* src[N];
  void* dst[N];
  long long count[N];
  int first[N + 1];  // chunks before
  uint32_t f32[(N + 31) / 32];
  int n, chunk;
};

struct Piece {
  const void* src;
  void* dst;
  long long at;  // first element
  int n;
  bool f32;
};

template <int N>
__device__ __forceinline__ Piece piece_of(const ClipTable<N>& tab, int c) {
  int lo = 0, hi = tab.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= c) lo = mid; else hi = mid - 1;
  }
  Piece p;
  p.src = tab.src[lo];
  p.dst = tab.dst[lo];
  p.at = static_cast<long long>(c - tab.first[lo]) * tab.chunk;
  p.n = static_cast<int>(min(static_cast<long long>(tab.chunk), tab.count[lo] - p.at));
  p.f32 = tab.f32[lo >> 5] >> (lo & 31) & 1u;
  return p;
}

__device__ __forceinline__ float value_of(const float* p, long long i) { return p[i]; }
__device__ __forceinline__ float value_of(const uint16_t* p, long long i) {
  return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}
__device__ __forceinline__ void put(float* p, long long i, float v) { p[i] = v; }
__device__ __forceinline__ void put(uint16_t* p, long long i, float v) {
  p[i] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xffffu);
}

// Sums of a CTA in which squares keep their bits: one below the normal numbers is off by
// 2^-150, 2^40 of them by less than the last place of 1e-25; and a few thousand sums of
// 1e30 stay finite.
__device__ __forceinline__ bool in_range(float s) { return s >= 1e-25f && s <= 1e30f; }

// This thread's share of a chunk's squares; *some: whether it has a value but 0.
template <typename T>
__device__ float squares_of(const T* __restrict__ p, int n, int tid, bool* some_out) {
  constexpr int W = 16 / sizeof(T);
  float s = 0.0f;
  uint32_t some = 0;
  const bool wide = (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
  const int nv = wide ? n / W : 0;
  const uint4* v = reinterpret_cast<const uint4*>(p);
  for (int i0 = 0; i0 < nv; i0 += 4 * kThreads) {
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * kThreads + tid;
      u[j] = i < nv ? __ldg(v + i) : make_uint4(0, 0, 0, 0);
    }
    float a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      some |= (u[j].x | u[j].y | u[j].z | u[j].w) & (sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu);  // -0 is 0
      a[j] = 0.0f;
      if constexpr (sizeof(T) == 2) {
        float f[8];
        unpack8(u[j], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[j] = fmaf(f[e], f[e], a[j]);
      } else {
        const float f[4] = {__uint_as_float(u[j].x), __uint_as_float(u[j].y), __uint_as_float(u[j].z),
                            __uint_as_float(u[j].w)};
#pragma unroll
        for (int e = 0; e < 4; ++e) a[j] = fmaf(f[e], f[e], a[j]);
      }
    }
    s += (a[0] + a[1]) + (a[2] + a[3]);
  }
  for (int i = nv * W + tid; i < n; i += kThreads) {
    const float f = value_of(p, i);
    some |= __float_as_uint(f) & 0x7fffffffu;
    s = fmaf(f, f, s);
  }
  *some_out = some != 0;
  return s;
}

template <typename T>
__device__ double squares_in_double(const T* __restrict__ p, int n, int tid) {
  double d = 0.0;
  for (int i = tid; i < n; i += kThreads) {
    const double f = value_of(p, i);
    d += f * f;
  }
  return d;
}

// hi + lo, lo being what the roundings of hi left: the next sum waits for hi alone.
struct alignas(8) Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair operator+(const Pair& a, const Pair& b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  return {s, ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo)};
}
__device__ __forceinline__ Pair exchanged(const Pair& v, int d) {
  return {__shfl_xor_sync(0xffffffffu, v.hi, d), __shfl_xor_sync(0xffffffffu, v.lo, d)};
}
__device__ __forceinline__ double exchanged(double v, int d) { return __shfl_xor_sync(0xffffffffu, v, d); }

// Sum over a CTA of NT threads, in its order; red: a value a warp.
template <int NT, typename T>
__device__ __forceinline__ T block_sum(T v, T* red) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v = v + exchanged(v, d);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[threadIdx.x & (NT / 32 - 1)];
#pragma unroll
  for (int d = NT / 64; d >= 1; d >>= 1) v = v + exchanged(v, d);
  return v;
}

// The CTAs' sums: pairs, and double (where the pair is out of range).
struct Parts {
  double* exact;
  Pair* sum;
};
__device__ __forceinline__ bool is_odd(const Pair& sum) { return sum.hi != 0.0f && !in_range(sum.hi); }

// Sum over the CTA of the squares of every `step`th chunk from `first` on (which may
// differ between its 256s of threads): a pair, or NaN where it is out of range, and then
// double.
struct Sum {
  Pair sum;
  double exact;
};
template <int NT, int N>
__device__ __forceinline__ Sum sum_chunks(const ClipTable<N>& tab, int first, int step) {
  __shared__ Pair red[NT / 32];
  __shared__ double red_exact[NT / 32];
  const int tid = threadIdx.x & (kThreads - 1);
  float s = 0.0f, lost = 0.0f;  // compensated
  bool any = false;
  for (int c = first; c < tab.first[tab.n]; c += step) {
    const Piece p = piece_of(tab, c);
    bool some;
    const float add = p.f32 ? squares_of(static_cast<const float*>(p.src) + p.at, p.n, tid, &some)
                            : squares_of(static_cast<const uint16_t*>(p.src) + p.at, p.n, tid, &some);
    any |= some;
    const float y = add - lost, t = s + y;
    lost = (t - s) - y;
    s = t;
  }
  const Pair sum = block_sum<NT>(Pair{s, -lost}, red);
  if (!__syncthreads_or(any) || in_range(sum.hi)) return {sum, 0.0};
  double d = 0.0;
  for (int c = first; c < tab.first[tab.n]; c += step) {
    const Piece p = piece_of(tab, c);
    d += p.f32 ? squares_in_double(static_cast<const float*>(p.src) + p.at, p.n, tid)
               : squares_in_double(static_cast<const uint16_t*>(p.src) + p.at, p.n, tid);
  }
  return {{__int_as_float(0x7fc00000), 0.0f}, block_sum<NT>(d, red_exact)};
}

template <int N>
__global__ void __launch_bounds__(kThreads) clip_norm_kernel(const __grid_constant__ ClipTable<N> tab, Parts parts) {
  griddep_launch_dependents();
  griddep_wait();
  const Sum s = sum_chunks<kThreads>(tab, blockIdx.x, gridDim.x);
  if (threadIdx.x == 0) {
    parts.sum[blockIdx.x] = s.sum;
    if (is_odd(s.sum)) parts.exact[blockIdx.x] = s.exact;
  }
}

// dst = src * by; a factor of 1 copies the bits (a product would give NaNs another payload).
template <typename T>
__device__ void scale_piece(const T* src, T* dst, int n, float by, int tid) {
  const bool copy = by == 1.0f;
  constexpr int W = 16 / sizeof(T);
  const bool wide = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15u) == 0;
  const int nv = wide ? n / W : 0;
  const uint4* v = reinterpret_cast<const uint4*>(src);
  uint4* o = reinterpret_cast<uint4*>(dst);
  for (int i0 = 0; i0 < nv; i0 += 4 * kThreads) {
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * kThreads + tid;
      if (i < nv) u[j] = v[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * kThreads + tid;
      if (i >= nv) continue;
      if (copy) {
        __stcs(o + i, u[j]);
        continue;
      }
      if constexpr (sizeof(T) == 2) {
        float f[8];
        unpack8(u[j], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= by;
        __stcs(o + i, pack8(f));
      } else {
        const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
        uint32_t r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = __float_as_uint(__uint_as_float(w[e]) * by);
        __stcs(o + i, make_uint4(r[0], r[1], r[2], r[3]));
      }
    }
  }
  for (int i = nv * W + tid; i < n; i += kThreads) {
    if (copy)
      dst[i] = src[i];
    else
      put(dst, i, value_of(src, i) * by);
  }
}

// The same where the factor is below fp32's normal numbers: it loses bits there, or all
// of them, which the products need not.
template <typename T>
__device__ void scale_piece_in_double(const T* src, T* dst, int n, double by, int tid) {
  for (int i = tid; i < n; i += kThreads) put(dst, i, static_cast<float>(value_of(src, i) * by));
}

// The norm and the factor; a norm that is not finite scales nothing.
struct Factor {
  float norm, by = 1.0f;
  bool far = false;    // by is not normal:
  double exact = 0.0;  // the factor then

  // Of a sum of squares that is in range, or 0.  By Newton's step for the root from what
  // its square leaves of the sum, and for the quotient from what the product leaves.
  __device__ __forceinline__ Factor(const Pair& sum, float max_norm) {
    const float r = sqrtf(sum.hi), inv = 1.0f / r;
    const float rest = r > 0.0f ? (fmaf(-r, r, sum.hi) + sum.lo) * (0.5f * inv) : 0.0f;
    norm = r + rest;
    if (!(norm > max_norm)) return;
    by = max_norm * inv;
    if (by < 2.0f * 1.175494351e-38f)
      in_double(static_cast<double>(r) + rest, max_norm);
    else
      by += (fmaf(-by, r, max_norm) - by * rest) * inv;
  }
  __device__ __forceinline__ Factor(double sum, float max_norm) {
    const double r = sqrt(sum);
    norm = static_cast<float>(r);
    if (norm > max_norm && norm <= 3.402823466e38f) in_double(r, max_norm);
  }

 private:
  __device__ __forceinline__ void in_double(double r, float max_norm) {
    const double f = max_norm / r;
    by = static_cast<float>(f);
    far = by < 1.175494351e-38f && max_norm > 0.0f;
    exact = f;
  }
};

template <int N>
__device__ __forceinline__ void scale_chunk(const ClipTable<N>& tab, int c, const Factor& f) {
  const Piece p = piece_of(tab, c);
  const int tid = threadIdx.x & (kThreads - 1);
  auto scale = [&](auto src, auto dst) {
    if (f.far)
      scale_piece_in_double(src + p.at, dst + p.at, p.n, f.exact, tid);
    else
      scale_piece(src + p.at, dst + p.at, p.n, f.by, tid);
  };
  if (p.f32)
    scale(static_cast<const float*>(p.src), static_cast<float*>(p.dst));
  else
    scale(static_cast<const uint16_t*>(p.src), static_cast<uint16_t*>(p.dst));
}

template <int N>
__global__ void __launch_bounds__(kThreads) clip_scale_kernel(const __grid_constant__ ClipTable<N> tab, Parts parts,
                                                              int P, float max_norm, int in_place,
                                                              float* __restrict__ norm) {
  __shared__ Pair red[kThreads / 32];
  __shared__ double red_exact[kThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  Pair s = {0.0f, 0.0f};
  bool odd = false;
  for (int i0 = threadIdx.x; i0 < P; i0 += 5 * kThreads) {
    Pair v[5];  // all on their way at once: up to 1280 sums in one round
#pragma unroll
    for (int j = 0; j < 5; ++j) v[j] = i0 + j * kThreads < P ? parts.sum[i0 + j * kThreads] : Pair{0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 5; ++j) {
      odd |= is_odd(v[j]);
      s = s + v[j];
    }
  }
  const bool any_odd = __syncthreads_or(odd);
  double d = 0.0;
  if (any_odd) {
    for (int i = threadIdx.x; i < P; i += kThreads) {
      const Pair v = parts.sum[i];
      d += is_odd(v) ? parts.exact[i] : static_cast<double>(v.hi) + v.lo;
    }
  }
  const Factor factor = any_odd ? Factor(block_sum<kThreads>(d, red_exact), max_norm)
                                : Factor(block_sum<kThreads>(s, red), max_norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = factor.norm;
  if (in_place && factor.by == 1.0f) return;
  for (int c = tab.first[tab.n] - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) scale_chunk(tab, c, factor);
}

template <int N>
__global__ void __launch_bounds__(kOneThreads) clip_one_kernel(const __grid_constant__ ClipTable<N> tab, float max_norm,
                                                               int in_place, float* __restrict__ norm) {
  __shared__ Pair sum;
  __shared__ double exact;
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kStep = kOneCtas * (kOneThreads / kThreads);
  const int first = (threadIdx.x / kThreads) * kOneCtas + blockIdx.x;
  const Sum own = sum_chunks<kOneThreads>(tab, first, kStep);
  if (threadIdx.x == 0) {
    sum = own.sum;
    exact = own.exact;
  }
  __syncwarp();
  cluster_sync_all();
  auto sum_of = [&](int c) {
    const uint32_t at = mapa_shared(smem_u32(&sum), c);
    Pair v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.hi), "=f"(v.lo) : "r"(at));
    return v;
  };
  Pair s = {0.0f, 0.0f};
  double d = 0.0;
  bool odd = false;
#pragma unroll
  for (int c = 0; c < kOneCtas; ++c) {
    const Pair v = sum_of(c);
    odd |= is_odd(v);
    s = s + v;
  }
  if (odd) {
    for (int c = 0; c < kOneCtas; ++c) {
      const Pair v = sum_of(c);
      double e;
      asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(e) : "r"(mapa_shared(smem_u32(&exact), c)));
      d += is_odd(v) ? e : static_cast<double>(v.hi) + v.lo;
    }
  }
  __syncwarp();
  cluster_sync_all();  // the other CTAs' sums have been read: none of them leaves before
  const Factor factor = odd ? Factor(d, max_norm) : Factor(s, max_norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = factor.norm;
  if (in_place && factor.by == 1.0f) return;
  for (int c = first; c < tab.first[tab.n]; c += kStep) scale_chunk(tab, c, factor);
}

constexpr int kSmallTable = 64, kLargeTable = 1000;  // 1.9 and 28.2 KB of parameters

// Chunks of one launch's tensors.
template <int N>
void fill(ClipTable<N>& tab, const ClipTensor* t, int n, int chunk) {
  tab.n = n;
  tab.chunk = chunk;
  for (uint32_t& w : tab.f32) w = 0;
  long long first = 0;
  for (int i = 0; i < n; ++i) {
    tab.src[i] = t[i].src;
    tab.dst[i] = t[i].dst;
    tab.count[i] = t[i].count;
    tab.first[i] = static_cast<int>(first);
    if (t[i].f32) tab.f32[i >> 5] |= 1u << (i & 31);
    first += (t[i].count + chunk - 1) / chunk;
  }
  tab.first[n] = static_cast<int>(first);
}

int grid_of(const int* first, int n, int most) { return first[n] < most ? (first[n] > 0 ? first[n] : 1) : most; }

template <int N>
cudaError_t run(const ClipTensor* t, int n, int chunk, float max_norm, int in_place, const Parts& parts, int most,
                float* norm, bool norm_only, bool over, cudaStream_t s) {
  int P = 0;
  ClipTable<N> tab;
  for (int i = 0; i == 0 || i < n; i += N) {
    fill<N>(tab, t + i, n - i < N ? n - i : N, chunk);
    const int grid = grid_of(tab.first, tab.n, most);
    const cudaError_t e = launch_short(over, clip_norm_kernel<N>, dim3(grid), dim3(kThreads), 0, s, tab,
                                       Parts{parts.exact + P, parts.sum + P});
    if (e != cudaSuccess) return e;
    P += grid;
  }
  for (int i = 0; i == 0 || i < n; i += N) {
    if (n > N) fill<N>(tab, t + i, n - i < N ? n - i : N, chunk);
    const int grid = norm_only ? 1 : grid_of(tab.first, tab.n, most);
    const cudaError_t e = launch_short(over, clip_scale_kernel<N>, dim3(grid), dim3(kThreads), 0, s, tab,
                                       parts, P, max_norm, in_place || norm_only, norm);
    if (e != cudaSuccess || norm_only) return e;
  }
  return cudaSuccess;
}

}  // namespace

namespace {
int clip_ctas(int sms) { return 8 * sms; }
int clip_launches(int n) { return n <= kSmallTable ? 1 : (n + kLargeTable - 1) / kLargeTable; }
}  // namespace

// What one cluster takes: 262144 values are 8 us of its device time.
constexpr int64_t kOneValues = 1 << 18;

size_t clip_scratch_bytes(int n, int64_t total, int sms) {
  if (n <= kSmallTable && total <= kOneValues) return 0;
  return static_cast<size_t>(clip_launches(n)) * clip_ctas(sms) * (sizeof(double) + sizeof(Pair));
}

cudaError_t launch_clip(const ClipTensor* t, int n, float max_norm, bool in_place, void* scratch, float* norm, int sms,
                        cudaStream_t stream) {
  long long total = 0;
  for (int i = 0; i < n; ++i) total += t[i].count;
  if (n <= kSmallTable && total <= kOneValues) {
    ClipTable<kSmallTable> tab;
    fill(tab, t, n, 4096);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kOneCtas);
    cfg.blockDim = dim3(kOneThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kOneCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, clip_one_kernel<kSmallTable>, tab, max_norm, static_cast<int>(in_place), norm);
  }
  Parts parts;
  parts.exact = static_cast<double*>(scratch);
  parts.sum = reinterpret_cast<Pair*>(parts.exact + static_cast<size_t>(clip_launches(n)) * clip_ctas(sms));
  // some eight chunks a CTA, of 4096 values at least and 32768 at most
  const int most = clip_ctas(sms);
  long long chunk = (total / (8LL * most) + 4095) / 4096 * 4096;
  chunk = chunk < 4096 ? 4096 : chunk > 32768 ? 32768 : chunk;
  const bool over = launch_over(6 * total, stream);  // two reads and a write
  const bool norm_only = max_norm > 3.402823466e38f && in_place;
  if (n <= kSmallTable)
    return run<kSmallTable>(t, n, static_cast<int>(chunk), max_norm, in_place, parts, most, norm, norm_only, over,
                            stream);
  return run<kLargeTable>(t, n, static_cast<int>(chunk), max_norm, in_place, parts, most, norm, norm_only, over,
                          stream);
}

}  // namespace gmm
