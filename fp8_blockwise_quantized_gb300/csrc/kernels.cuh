// Kernel entry points and their host-side launchers (internal to the library).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <utility>

#include "common.cuh"

namespace gmm {

// Launch with programmatic stream serialization (see griddep_wait): the kernel
// may start while the previous kernel on the stream finishes.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The same for short calls: programmatic serialization (`over`) only where it gains
// more than it costs.  It hides 2 to 4 us between two kernels of one stream, and its
// launch takes 1.5 to 2 us more of the host's time, which is what bounds a call of a
// few microseconds (router of 16 tokens through the Python entry point: 11.5 us with
// it, 10.7 without).
template <typename... KArgs, typename... Args>
cudaError_t launch_short(bool over, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                         Args&&... args) {
  if (over) return launch_pdl(kernel, grid, block, smem, stream, std::forward<Args>(args)...);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}
// Whether it does: from 32 MB on (5 us of HBM traffic), and in a captured graph, whose
// launches cost the host nothing.
inline bool launch_over(long long bytes, cudaStream_t stream) {
  if (bytes >= 32LL << 20) return true;
  if (stream == nullptr) return false;  // the legacy stream cannot be captured
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  return cudaStreamIsCapturing(stream, &status) == cudaSuccess && status == cudaStreamCaptureStatusActive;
}

// Raises a kernel's dynamic shared memory limit once per device (`done`: one
// bit per device, a static of the calling launcher).
template <typename... KArgs>
cudaError_t allow_smem(void (*kernel)(KArgs...), int smem, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// ---- a1 metadata ------------------------------------------------------------
__global__ void group_metadata_kernel(const int32_t* sizes, int G, int M, int32_t* ws, Tile* tiles,
                                      int32_t* order, Tile* pair_tiles);
// Launches the metadata kernel into a workspace laid out for (G, M).
cudaError_t launch_group_metadata(const int32_t* sizes, int G, int M, void* workspace, cudaStream_t stream);

// ---- a2 / a3 quantization -----------------------------------------------------
constexpr int kLhsBlocksPerWarp = 8;
__global__ void quantize_lhs_kernel(const uint4* x, int M, int KB, long long nblocks, uint2* xq, float* xs);
__global__ void quantize_rhs_kernel(const uint16_t* w, int K, int N, uint8_t* wq, float* ws);
__global__ void quantize_rhs_w4_kernel(const uint16_t* w, int K, int N, uint8_t* wq4, float* ws);

// ---- grouped GEMMs ------------------------------------------------------------
// Arguments shared by the grouped forward kernels.
struct FwdArgs {
  const float* xs;        // fp32 [K/128][M] (FP8 only)
  const float* ws;        // fp32 [G][K/128][Nw/128] (FP8 only)
  const int32_t* meta;    // workspace words
  const Tile* tiles;      // workspace tile list (128-row tiles)
  const Tile* pair_tiles; // workspace 256-row tiles (CTA-pair FP8 kernel)
  uint16_t* out;          // bf16 [M][N] (may be null with hq)
  uint8_t* hq;            // fused quantized output: e4m3 [M][N] (null: none)
  float* hs;              // fused quantized output scales: fp32 [N/128][M]
  int M, K, N;            // N = output columns
  int fuse;               // 1: silu(gate) * up, W has 2N columns
  int bn;                 // FP8: columns of W per unit (0: by N)
  int col_major;          // FP8: units ordered column block major
  int b_fmt;              // FP8: weight code type in the MMA instruction descriptor
                          // (kind::f8f6f4: 0 = e4m3, 5 = e2m1)
  int stages;             // FP8: ring slots of the launched instance
  int tmem_bufs;          // FP8: TMEM partial buffers of the launched instance
  uint64_t wait_limit_ns;
};

struct TgmmArgs {
  const int32_t* meta;    // workspace words (offsets)
  const int32_t* order;   // workspace: groups by size, descending
  uint16_t* dw;           // bf16 [G][K][N]
  int G, M, K, N;
  int stages;             // CTA-pair kernel with 256-column units: ring slots (4..6)
  int claim_ahead;        // CTA-pair kernel: units claimed beyond the producer (1..12)
  int max_batch;          // CTA-pair kernel: most small units per claim (1..4)
  uint64_t wait_limit_ns;
  const float* xs;        // 8-bit checkpoint: fp32 [K/128][M] scales of x's codes
  const float* parts;     // 8-bit checkpoint, splits > 1: the parts' sums, fp32 [splits][G][K][N]
  int splits;             // parts that each group's rows are cut into
  const int32_t* sizes;   // 8-bit checkpoint: group_sizes, G <= kScanGroups, or NULL: the metadata is in the workspace
  const Tile* tiles;      // 8-bit checkpoint: workspace tile list, filled when sizes is given
};

// The gated feed-forward block's kernels: the forward (K = columns of x) and
// the backward (K = columns of dy, the reduction of dh = dy W2^T).
struct SwigluArgs {
  const int32_t* meta;    // workspace words
  const Tile* tiles;      // workspace tile list (128-row tiles)
  const int32_t* sizes;   // group_sizes, G <= kScanGroups, or NULL: the metadata is in the workspace
  uint16_t* h;            // bf16 [M][N] (backward: may be null)
  uint16_t* gu;           // kept gate | up, bf16 [M][2N], or null:
  uint8_t* guq;           // e4m3 codes [M][2N] with
  float* gus;             // fp32 [2N/128][M] scales
  uint16_t* dgu;          // backward: gradient of gate | up, bf16 [M][2N]
  int G, M, K, N;
  uint64_t wait_limit_ns;
};

struct Mx4Args {
  const int32_t* meta;    // workspace words
  const Tile* tiles;      // workspace tile list (128-row tiles)
  const int32_t* sizes;   // group_sizes, G <= kScanGroups, or NULL: the metadata is in the workspace
  const uint32_t* xs;     // E8M0 scales of x, words of four blocks [K/128][M]
  const uint8_t* ws;      // E8M0 scales of w, tiles [G][Nw/128][K/128][512]
  uint16_t* out;          // bf16 [M][N] (may be null with hq)
  uint8_t* hq;            // MXFP4 output: codes [M][N/2] (null: none)
  uint32_t* hs;           // and scale words [N/128][M]
  int G, M, K, N;         // N = output columns
  int fuse;               // 1: silu(gate) * up, w has 2N columns
  int bn;                 // weight columns per unit (128 or 256)
  uint64_t wait_limit_ns;
};

// Host launchers: `grid` CTAs (persistent), on `stream`.  Return the launch error.
// map_out: the bf16 output (out, or h when fused) [M, N], box 64 columns x
// 32 rows, 128-byte swizzle; read only when args.out is not null.
cudaError_t launch_gmm_fp8(const CUtensorMap& map_a, const CUtensorMap& map_b, const CUtensorMap& map_out,
                           const FwdArgs& args, int grid, cudaStream_t stream);
// The single-CTA kernel's BN = 128 instances (gmm_fp8_n128.cu).
cudaError_t launch_gmm_fp8_n128(const CUtensorMap& map_a, const CUtensorMap& map_b, const CUtensorMap& map_out,
                                const FwdArgs& args, int grid, cudaStream_t stream);
// The CTA-pair FP8 kernel: map_b's box is 64 rows (half of a 128-column MMA
// half); at most max_pairs clusters of two CTAs.
cudaError_t launch_gmm_fp8_pair(const CUtensorMap& map_a, const CUtensorMap& map_b, const CUtensorMap& map_out,
                                const FwdArgs& args, int max_pairs, cudaStream_t stream);
cudaError_t launch_gmm_bf16(const CUtensorMap& map_a, const CUtensorMap& map_b, const FwdArgs& args, int grid,
                            cudaStream_t stream);
// bf16 dgrad: the forward kernel with a K-major weight ([G*N_out, K] view);
// args.K = reduction length, args.N = output columns.
cudaError_t launch_gmm_bf16_dgrad(const CUtensorMap& map_a, const CUtensorMap& map_b, const FwdArgs& args,
                                  int grid, cudaStream_t stream);
cudaError_t launch_tgmm_bf16(const CUtensorMap& map_x, const CUtensorMap& map_dy, const CUtensorMap& map_dw,
                             const TgmmArgs& args, int grid, cudaStream_t stream);

// map_x: x [M, K], box 64 x 128; map_w: w [G*K, 2N], box 64 x 64.
cudaError_t launch_gmm_swiglu_fwd(const CUtensorMap& map_x, const CUtensorMap& map_w, const SwigluArgs& args,
                                  int grid, cudaStream_t stream);
// map_dy: dy [M, K], box 64 x 128; map_w2: w2 [G*N, K], box 64 x 128.
cudaError_t launch_gmm_swiglu_bwd(const CUtensorMap& map_dy, const CUtensorMap& map_w2, const SwigluArgs& args,
                                  int grid, cudaStream_t stream);
// map_x: codes [M, K] bytes, box 128 x 64; map_dy: box 64 x 64; map_dw: dw [G*K, N], box 64 x 32, or with
// splits > 1 the parts [splits*G*K, N], box 32 x 32.
cudaError_t launch_tgmm_ckpt(const CUtensorMap& map_x, const CUtensorMap& map_dy, const CUtensorMap& map_dw,
                             const TgmmArgs& args, int max_pairs, cudaStream_t stream);

int tgmm_ckpt_splits(int G, int64_t M, int64_t K, int64_t N, int sms);

// ---- MXFP4 --------------------------------------------------------------------
__global__ void mx4_quantize_lhs_kernel(const uint4* x, int M, uint32_t KB, uint32_t steps, uint32_t* xq,
                                        uint32_t* xs);
__global__ void mx4_quantize_rhs_kernel(const uint16_t* w, int K, int N, uint8_t* wq, uint8_t* ws);
// map_a: codes [M, K/2] bytes, box 128 x 128; map_b: codes [G*Nw, K/2] bytes,
// box 128 x bn (bn / 2 when fused); map_out: out [M, N], box 64 x 32.
cudaError_t launch_gmm_mx4(const CUtensorMap& map_a, const CUtensorMap& map_b, const CUtensorMap& map_out,
                           const Mx4Args& args, int grid, cudaStream_t stream);

// ---- the layer around the experts: router, sorted rows, norms, clipping --------
struct RouteArgs {
  const void* logits;      // fp32 or bf16 [T][E]
  const float* bias;       // [E] or null (forward)
  const float* dweights;   // [T][k] (backward)
  const int32_t* ids;      // [T][k] (backward)
  int32_t* ids_out;        // forward
  float* weights;          // [T][k], forward
  void* dlogits;           // [T][E], backward
  long long T;
  int E, k;
  int f32, softmax, renorm;
  float scale;
};
cudaError_t launch_route(const RouteArgs& args, cudaStream_t stream);
cudaError_t launch_route_bwd(const RouteArgs& args, cudaStream_t stream);

// Device bytes that the sort of N ids needs besides its outputs (0: none).
size_t sort_scratch_bytes(int64_t N, int G);
cudaError_t launch_sort_rows(const int32_t* ids, int64_t N, int G, int32_t* rows, int32_t* sizes, void* scratch,
                             cudaStream_t stream);
// T tokens of K columns, k choices each; M = T * k sorted rows.
cudaError_t launch_gather_rows(const void* x, const int32_t* rows, int64_t T, int k, int64_t K, void* out,
                               cudaStream_t stream);
cudaError_t launch_gather_quantize(const void* x, const int32_t* rows, int64_t T, int k, int64_t K, void* xq, float* xs,
                                   cudaStream_t stream);
cudaError_t launch_gather_mx4(const void* x, const int32_t* rows, int64_t T, int k, int64_t K, void* xq, void* xs,
                              cudaStream_t stream);
cudaError_t launch_combine_rows(const void* y, const int32_t* rows, const float* weights, int64_t T, int k, int64_t K,
                                void* out, cudaStream_t stream);
cudaError_t launch_combine_rows_bwd(const void* dout, const void* y, const int32_t* rows, const float* weights,
                                    int64_t T, int k, int64_t K, void* dy, float* dweights, int sms,
                                    cudaStream_t stream);

struct NormJoinArgs {
  const void* x;              // residual stream [T][K], fp32 or bf16
  const uint16_t* b;          // the block's output, bf16 [T][K], or null
  const float* w_post;        // [K] or null
  const float* gate_col;      // [K] or null
  const uint16_t* gate_full;  // bf16 [T][K] or null
  const float* w_next;        // [K] or null
  void* out;                  // as x; written when b is given
  uint16_t* n;                // bf16 [T][K]; written when w_next is given
  long long T;
  int K, f32;
  int row_threads;            // set by the launcher
  float alpha, beta, eps;
};
struct NormJoinBwdArgs {
  const void* dout;           // as out, or null
  const uint16_t* dn;         // bf16 [T][K] or null
  const void* out;            // the forward's out (its x without a block); read when dn is given
  const uint16_t* b;
  const float* w_post;
  const float* gate_col;
  const uint16_t* gate_full;
  const float* w_next;
  void* dx;                   // as out, or null
  uint16_t* db;               // bf16 [T][K] (with b)
  float* dw_post;             // [K] or null
  float* dgate_col;           // [K] or null
  uint16_t* dgate_full;       // bf16 [T][K] (with gate_full)
  float* dw_next;             // [K] or null
  float* parts;               // [norm_join_parts][2][K]
  long long T;
  int K, f32;
  int row_threads;            // set by the launcher
  float alpha, beta, eps;
};
cudaError_t launch_norm_join(const NormJoinArgs& args, int sms, cudaStream_t stream);
int norm_join_parts(int64_t T, int64_t K, int sms);
cudaError_t launch_norm_join_bwd(const NormJoinBwdArgs& args, int sms, cudaStream_t stream);

struct ClipTensor {
  const void* src;
  void* dst;
  int64_t count;
  int f32;
};
size_t clip_scratch_bytes(int n, int64_t total, int sms);
cudaError_t launch_clip(const ClipTensor* t, int n, float max_norm, bool in_place, void* scratch, float* norm, int sms,
                        cudaStream_t stream);

// Tile geometry the host needs to build tensor maps and size grids.
struct Fp8Geometry {
  int bn_mma;      // MMA N (columns of W per stage)
  int out_cols;    // output columns per work unit
  int b_box_rows;  // rows of the W tensor-map box
};
Fp8Geometry fp8_geometry(int N, int fuse, int bn = 0);
Fp8Geometry bf16_geometry(int N, int fuse);
int tgmm_bn(int N);

}  // namespace gmm
