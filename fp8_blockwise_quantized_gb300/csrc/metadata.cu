// a1: group metadata on the device.
//
// Rows are sorted by expert into contiguous groups ("MoE 优化的探索", §3.7.2);
// a grouped kernel finds each tile's expert through offsets and a tile list
// built from group_sizes on the device ("实现差距：GMM Kernel（V1 vs V2）", §1
// and §2.2: the metadata is filled inside the kernel, not on the host).
//
// One CTA of 1024 threads: each thread owns a contiguous run of at most
// ceil(G/1024) groups, the block scans the per-thread row and tile counts, and
// every thread then writes its groups' offsets, 128-row tiles and 256-row
// tiles (the row tiles of the CTA-pair FP8 kernel).
#include "common.cuh"
#include "kernels.cuh"
#include "metadata.cuh"
#include "ptx.cuh"

namespace gmm {

__global__ void __launch_bounds__(1024) group_metadata_kernel(const int32_t* __restrict__ sizes, int G,
                                                                int M, int32_t* __restrict__ ws,
                                                                Tile* __restrict__ tiles,
                                                                int32_t* __restrict__ order,
                                                                Tile* __restrict__ pair_tiles) {
  __shared__ long long warp_sums[33];
  __shared__ unsigned long long keys[kMaxGroups];
  griddep_launch_dependents();
  griddep_wait();  // group_sizes may come from the previous kernel
  write_group_metadata<32>(sizes, G, M, ws, tiles, order, pair_tiles, threadIdx.x, warp_sums, keys, true,
                           [] { __syncthreads(); });
}

cudaError_t launch_group_metadata(const int32_t* sizes, int G, int M, void* workspace, cudaStream_t stream) {
  char* base = static_cast<char*>(workspace);
  return launch_pdl(group_metadata_kernel, dim3(1), dim3(1024), 0, stream, sizes, G, M, static_cast<int32_t*>(workspace),
                    reinterpret_cast<Tile*>(base + tiles_offset_bytes(G)),
                    reinterpret_cast<int32_t*>(base + order_offset_bytes(G, M)),
                    reinterpret_cast<Tile*>(base + pair_tiles_offset_bytes(G, M)));
}

}  // namespace gmm
