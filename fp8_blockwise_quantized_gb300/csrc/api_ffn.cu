// Host side of the feed-forward block's entry points (include/gmm.h): the
// gated forward and backward, the weight gradient from 8-bit checkpoints and
// the MXFP4 quantisation and products.  Nothing here allocates device memory
// or synchronizes.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gmm.h"
#include "common.cuh"
#include "host.cuh"
#include "kernels.cuh"
#include "metadata.cuh"

using namespace gmm;

namespace {

// every pointer 16-byte aligned (NULL passes)
template <typename... P>
bool all_aligned(P... p) {
  return (((reinterpret_cast<uintptr_t>(p) & 15u) == 0) && ...);
}

const Tile* tiles_of(const void* workspace, int G) {
  return reinterpret_cast<const Tile*>(static_cast<const char*>(workspace) + tiles_offset_bytes(G));
}

// Upper bound of the row tiles: every group adds at most one that is not
// full, and none without rows.
long long max_tiles(int G, int64_t M) { return (M + kBM - 1) / kBM + (M < G ? M : G); }

// Whether a kernel that can reads the sizes itself: no metadata launch.
bool scanned(const int32_t* group_sizes, int G, int64_t M) { return group_sizes && G <= kScanGroups && M > 0; }

// The device, the workspace and (unless group_sizes is NULL) the metadata.
gmm_status begin(const int32_t* group_sizes, int G, int64_t M, void* workspace, size_t workspace_bytes,
                 cudaStream_t s, int* sms) {
  gmm_status st = host_check_workspace(workspace, workspace_bytes, G, M);
  if (st != GMM_OK) return st;
  if ((st = host_device_sms(sms)) != GMM_OK) return st;
  return group_sizes ? host_launch_metadata(group_sizes, G, M, workspace, s) : GMM_OK;
}

gmm_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? GMM_OK : host_cuda_fail(e, what); }

// One CTA per unit up to one per SM, and one without a unit, if there is room,
// for the CTA that fills the workspace when the kernel reads the sizes itself.
int grid_of(long long units, const int32_t* sizes, int sms) {
  if (sizes) ++units;
  return static_cast<int>(units < sms ? units : sms);
}

// The kernels' unit indices are 32-bit, with the grid's claims on top.
constexpr long long kMaxUnits = 1LL << 30;

constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr CUtensorMapDataType kByte = CU_TENSOR_MAP_DATA_TYPE_UINT8;

// The kept gate | up values: bf16 (gu) or e4m3 with scales (guq, gus), one of them.
gmm_status check_kept(int64_t M, const void* gu, const void* guq, const float* gus) {
  if (M == 0) return GMM_OK;
  const bool e4m3 = guq || gus;
  if (e4m3 ? (!guq || !gus) : !gu) return GMM_ERR_NULL;
  return gu && e4m3 ? GMM_ERR_UNSUPPORTED : GMM_OK;
}

gmm_status mx4_entry(const void* xq, const void* xs, const void* wq, const void* ws, const int32_t* group_sizes, int G,
                     int64_t M, int64_t K, int64_t N, int fuse, void* out, void* hq, void* hs, bool quant,
                     void* workspace, size_t workspace_bytes, void* stream) {
  const int64_t Nw = fuse ? 2 * N : N;
  gmm_status st = host_check_grouped(G, M, K, N, Nw);
  if (st != GMM_OK) return st;
  if (!wq || !ws) return GMM_ERR_NULL;
  if (M > 0 && (!xq || !xs || (quant ? (!hq || !hs) : !out))) return GMM_ERR_NULL;
  if (!all_aligned(xq, xs, wq, ws, group_sizes, out, hq, hs)) return GMM_ERR_ALIGN;
  if (max_tiles(G, M) * (N / 64) > kMaxUnits) return GMM_ERR_SHAPE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int sms = 0;
  const int32_t* sizes = scanned(group_sizes, G, M) ? group_sizes : nullptr;
  if ((st = begin(sizes ? nullptr : group_sizes, G, M, workspace, workspace_bytes, s, &sms)) != GMM_OK) return st;
  if (M == 0) return GMM_OK;
  // 128-column units while one per SM covers the call: latency (8 row tiles, K
  // 2048, N 2 x 512: 8.4 us, 9.2 with 256; 128 units of K 512: 6.3 and 6.5).
  // Beyond that 256: half the reads of x (256 units of 128 columns: 11.4 to
  // 15.0 us, 128 of 256: 9.9 to 11.8).
  const int bn = (fuse || N % 256 == 0) && max_tiles(G, M) * (Nw / 128) > sms ? 256 : 128;
  CUtensorMap map_a, map_b, map_out;
  if ((st = host_encode_2d(&map_a, kByte, 1, xq, K / 2, M, 128, 128)) != GMM_OK) return st;
  if ((st = host_encode_2d(&map_b, kByte, 1, wq, K / 2, G * Nw, 128, fuse ? bn / 2 : bn)) != GMM_OK) return st;
  if (out) {
    if ((st = host_encode_2d(&map_out, kBf16, 2, out, N, M, 64, 32)) != GMM_OK) return st;
  } else {
    map_out = map_a;  // never read
  }
  Mx4Args a{};
  a.meta = static_cast<const int32_t*>(workspace);
  a.tiles = tiles_of(workspace, G);
  a.sizes = sizes;
  a.G = G;
  a.xs = static_cast<const uint32_t*>(xs);
  a.ws = static_cast<const uint8_t*>(ws);
  a.out = static_cast<uint16_t*>(out);
  a.hq = quant ? static_cast<uint8_t*>(hq) : nullptr;
  a.hs = quant ? static_cast<uint32_t*>(hs) : nullptr;
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.N = static_cast<int>(N);
  a.fuse = fuse;
  a.bn = bn;
  a.wait_limit_ns = host_wait_limit_ns();
  const long long units = max_tiles(G, M) * (Nw / bn);
  return launched(launch_gmm_mx4(map_a, map_b, map_out, a, grid_of(units, sizes, sms), s),
                  "gmm_mx4 kernel launch");
}

}  // namespace

extern "C" {

gmm_status gmm_bf16_swiglu_fwd(const void* x, const void* w, const int32_t* group_sizes, int G, int64_t M, int64_t K,
                               int64_t N, void* h, void* gu, void* guq, float* gus, void* workspace,
                               size_t workspace_bytes, void* stream) {
  gmm_status st = host_check_grouped(G, M, K, N, 2 * N);
  if (st != GMM_OK) return st;
  if (!w || (M > 0 && (!x || !h))) return GMM_ERR_NULL;
  if ((st = check_kept(M, gu, guq, gus)) != GMM_OK) return st;
  if (!all_aligned(x, w, group_sizes, h, gu, guq, gus)) return GMM_ERR_ALIGN;
  const long long units = max_tiles(G, M) * (N / 64);  // narrow ones
  if (units > kMaxUnits) return GMM_ERR_SHAPE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int sms = 0;
  const int32_t* sizes = scanned(group_sizes, G, M) ? group_sizes : nullptr;
  if ((st = begin(sizes ? nullptr : group_sizes, G, M, workspace, workspace_bytes, s, &sms)) != GMM_OK) return st;
  if (M == 0) return GMM_OK;
  CUtensorMap map_x, map_w;
  if ((st = host_encode_2d(&map_x, kBf16, 2, x, K, M, 64, 128)) != GMM_OK) return st;
  if ((st = host_encode_2d(&map_w, kBf16, 2, w, 2 * N, G * K, 64, 64)) != GMM_OK) return st;
  SwigluArgs a{};
  a.meta = static_cast<const int32_t*>(workspace);
  a.tiles = tiles_of(workspace, G);
  a.sizes = sizes;
  a.G = G;
  a.h = static_cast<uint16_t*>(h);
  a.gu = static_cast<uint16_t*>(gu);
  a.guq = static_cast<uint8_t*>(guq);
  a.gus = gus;
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.N = static_cast<int>(N);
  a.wait_limit_ns = host_wait_limit_ns();
  return launched(launch_gmm_swiglu_fwd(map_x, map_w, a, grid_of(units, sizes, sms), s),
                  "gmm_swiglu forward launch");
}

gmm_status gmm_bf16_swiglu_bwd(const void* dy, const void* w2, const void* gu, const void* guq, const float* gus,
                               const int32_t* group_sizes, int G, int64_t M, int64_t K, int64_t N, void* dgu, void* h,
                               void* workspace, size_t workspace_bytes, void* stream) {
  gmm_status st = host_check_grouped(G, M, K, N, 2 * N);
  if (st != GMM_OK) return st;
  if (!w2 || (M > 0 && (!dy || !dgu))) return GMM_ERR_NULL;
  if ((st = check_kept(M, gu, guq, gus)) != GMM_OK) return st;
  if (!all_aligned(dy, w2, gu, guq, gus, group_sizes, dgu, h)) return GMM_ERR_ALIGN;
  const long long units = max_tiles(G, M) * (N / 128);  // narrow ones
  if (units > kMaxUnits) return GMM_ERR_SHAPE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int sms = 0;
  const int32_t* sizes = scanned(group_sizes, G, M) ? group_sizes : nullptr;
  if ((st = begin(sizes ? nullptr : group_sizes, G, M, workspace, workspace_bytes, s, &sms)) != GMM_OK) return st;
  if (M == 0) return GMM_OK;
  CUtensorMap map_dy, map_w2;
  if ((st = host_encode_2d(&map_dy, kBf16, 2, dy, K, M, 64, 128)) != GMM_OK) return st;
  if ((st = host_encode_2d(&map_w2, kBf16, 2, w2, K, G * N, 64, 128)) != GMM_OK) return st;
  SwigluArgs a{};
  a.meta = static_cast<const int32_t*>(workspace);
  a.tiles = tiles_of(workspace, G);
  a.sizes = sizes;
  a.G = G;
  a.h = static_cast<uint16_t*>(h);
  a.gu = static_cast<uint16_t*>(const_cast<void*>(gu));
  a.guq = static_cast<uint8_t*>(const_cast<void*>(guq));
  a.gus = const_cast<float*>(gus);
  a.dgu = static_cast<uint16_t*>(dgu);
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.N = static_cast<int>(N);
  a.wait_limit_ns = host_wait_limit_ns();
  return launched(launch_gmm_swiglu_bwd(map_dy, map_w2, a, grid_of(units, sizes, sms), s),
                  "gmm_swiglu backward launch");
}

size_t tgmm_fp8_ckpt_scratch_bytes(int G, int64_t M, int64_t K, int64_t N) {
  int sms = 0;
  if (host_check_grouped(G, M, K, N, N) != GMM_OK || host_device_sms(&sms) != GMM_OK) return 0;
  const int splits = tgmm_ckpt_splits(G, M, K, N, sms);
  return splits > 1 ? static_cast<size_t>(splits) * G * K * N * sizeof(float) : 0;
}

gmm_status tgmm_fp8_ckpt(const void* xq, const float* xs, const void* dy, const int32_t* group_sizes, int G, int64_t M,
                         int64_t K, int64_t N, void* dw, void* scratch, size_t scratch_bytes, void* workspace,
                         size_t workspace_bytes, void* stream) {
  gmm_status st = host_check_grouped(G, M, K, N, N);
  if (st != GMM_OK) return st;
  const long long tiles = static_cast<long long>(G) * ((K + 255) / 256) * ((N + 255) / 256);
  if (tiles > kMaxUnits) return GMM_ERR_SHAPE;
  if (!dw || (M > 0 && (!xq || !xs || !dy))) return GMM_ERR_NULL;
  if (!all_aligned(xq, xs, dy, group_sizes, dw, scratch)) return GMM_ERR_ALIGN;
  if ((st = host_check_workspace(workspace, workspace_bytes, G, M)) != GMM_OK) return st;
  int sms = 0;
  if ((st = host_device_sms(&sms)) != GMM_OK) return st;
  const int splits = scratch ? tgmm_ckpt_splits(G, M, K, N, sms) : 1;
  if (splits > 1 && scratch_bytes < static_cast<size_t>(splits) * G * K * N * sizeof(float)) return GMM_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int32_t* sizes = scanned(group_sizes, G, M) ? group_sizes : nullptr;
  if ((st = begin(sizes ? nullptr : group_sizes, G, M, workspace, workspace_bytes, s, &sms)) != GMM_OK) return st;
  // With M == 0 every group is empty: the kernel only writes zeros and never
  // reads x or dy, so the maps may describe a dummy one-row tensor.
  CUtensorMap map_x, map_dy, map_dw;
  if ((st = host_encode_2d(&map_x, kByte, 1, M > 0 ? xq : dw, K, M, 128, 64)) != GMM_OK) return st;
  if ((st = host_encode_2d(&map_dy, kBf16, 2, M > 0 ? dy : dw, N, M, 64, 64)) != GMM_OK) return st;
  st = splits > 1 ? host_encode_2d(&map_dw, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, scratch, N,
                                   static_cast<uint64_t>(splits) * G * K, 32, 32)
                  : host_encode_2d(&map_dw, kBf16, 2, dw, N, G * K, 64, 32);
  if (st != GMM_OK) return st;
  TgmmArgs a{};
  a.meta = static_cast<const int32_t*>(workspace);
  a.order = reinterpret_cast<const int32_t*>(static_cast<const char*>(workspace) + order_offset_bytes(G, M));
  a.dw = static_cast<uint16_t*>(dw);
  a.xs = xs;
  a.parts = static_cast<const float*>(scratch);
  a.splits = splits;
  a.sizes = sizes;
  a.tiles = tiles_of(workspace, G);
  a.G = G;
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.N = static_cast<int>(N);
  a.wait_limit_ns = host_wait_limit_ns();
  const long long units = tiles * splits;
  const int max_pairs = static_cast<int>(units < sms / 2 ? units : sms / 2);
  return launched(launch_tgmm_ckpt(map_x, map_dy, map_dw, a, max_pairs, s), "tgmm_ckpt kernel launch");
}

gmm_status gmm_mx4_quantize_lhs(const void* x, int64_t M, int64_t K, void* xq, void* xs, void* stream) {
  if (M < 0 || M > INT32_MAX || K < 128 || K % 128 != 0 || K > (1 << 24)) return GMM_ERR_SHAPE;
  if (M == 0) return GMM_OK;
  if (!x || !xq || !xs) return GMM_ERR_NULL;
  if (!all_aligned(x, xq, xs)) return GMM_ERR_ALIGN;
  int sms = 0;
  gmm_status st = host_device_sms(&sms);
  if (st != GMM_OK) return st;
  const long long steps = (M + 7) / 8 * (K / 128);  // a warp each, 8 warps per CTA
  if (steps >= (1LL << 31)) return GMM_ERR_SHAPE;   // 4 TB of x
  long long grid = (steps + 7) / 8;
  // many short CTAs: with an earlier form of the kernel, 65536 x 2048 took 59.8
  // us with 32 per SM, 63.4 with 16, 67.0 with 8 and 64.5 with one step a warp
  if (grid > static_cast<long long>(sms) * 32) grid = static_cast<long long>(sms) * 32;
  return launched(launch_pdl(mx4_quantize_lhs_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0,
                             static_cast<cudaStream_t>(stream), static_cast<const uint4*>(x), static_cast<int>(M),
                             static_cast<uint32_t>(K / 128), static_cast<uint32_t>(steps), static_cast<uint32_t*>(xq),
                             static_cast<uint32_t*>(xs)),
                  "mx4_quantize_lhs_kernel launch");
}

gmm_status gmm_mx4_quantize_rhs(const void* w, int G, int64_t K, int64_t N, void* wq, void* ws, void* stream) {
  if (G < 1 || K < 128 || K % 128 != 0 || N < 128 || N % 128 != 0 || K > (1 << 24) || N > (1 << 24))
    return GMM_ERR_SHAPE;
  const int64_t grid = static_cast<int64_t>(G) * (K / 128) * (N / 128);
  if (grid > INT32_MAX) return GMM_ERR_SHAPE;
  if (!w || !wq || !ws) return GMM_ERR_NULL;
  if (!all_aligned(w, wq, ws)) return GMM_ERR_ALIGN;
  int sms = 0;
  gmm_status st = host_device_sms(&sms);
  if (st != GMM_OK) return st;
  mx4_quantize_rhs_kernel<<<static_cast<unsigned>(grid), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(w), static_cast<int>(K), static_cast<int>(N), static_cast<uint8_t*>(wq),
      static_cast<uint8_t*>(ws));
  return launched(cudaGetLastError(), "mx4_quantize_rhs_kernel launch");
}

gmm_status gmm_mx4_fwd(const void* xq, const void* xs, const void* wq, const void* ws, const int32_t* group_sizes,
                       int G, int64_t M, int64_t K, int64_t N, int fuse_silu_mul, void* out, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return mx4_entry(xq, xs, wq, ws, group_sizes, G, M, K, N, fuse_silu_mul ? 1 : 0, out, nullptr, nullptr, false,
                   workspace, workspace_bytes, stream);
}

gmm_status gmm_mx4_fwd_swiglu_quant(const void* xq, const void* xs, const void* wq, const void* ws,
                                    const int32_t* group_sizes, int G, int64_t M, int64_t K, int64_t N, void* h,
                                    void* hq, void* hs, void* workspace, size_t workspace_bytes, void* stream) {
  return mx4_entry(xq, xs, wq, ws, group_sizes, G, M, K, N, 1, h, hq, hs, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
