// Work units of the persistent grouped kernels that claim their units as they
// go: a CTA's scheduler warp resolves each unit and hands it to the other
// roles through a queue in shared memory.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace gmm {

constexpr int kClaimSlots = 4;  // entries of a CTA's unit queue

// The queue of one CTA.  An entry is {g, row0, row1, column block}; g < 0:
// no more units.  READERS roles (warps, or single threads) take the entries
// in order and free each one they have read.
struct ClaimQueue {
  uint64_t* full;
  uint64_t* empty;
  int4* data;
  static constexpr int kBarriers = 2 * kClaimSlots;
  __device__ void init(int readers) const {
    for (int q = 0; q < kClaimSlots; ++q) {
      mbar_init(&full[q], 1);
      mbar_init(&empty[q], readers);
    }
  }
  __device__ bool get(uint32_t i, int4& e, bool warp_wide, int lane, volatile int* abort_word, uint64_t lim) const {
    const uint32_t slot = i % kClaimSlots, ph = (i / kClaimSlots) & 1u;
    bool ok = mbar_wait(&full[slot], ph, abort_word, lim);
    if (warp_wide) ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    e = data[slot];
    if (warp_wide) __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    return true;
  }
  // Scheduler (one thread): the CTA's first unit is its block index, the next
  // ones are claimed from the workspace counter, one claim in flight while the
  // current unit is published (a CTA that runs slower takes fewer units).
  // Unit u is row tile u / per_tile, column block u % per_tile.
  __device__ void schedule(const Tile* tiles, int* claimed, uint32_t num_units, uint32_t per_tile,
                           volatile int* abort_word, uint64_t lim) const {
    uint32_t u = blockIdx.x;
    for (uint32_t i = 0;; ++i) {
      const bool live = u < num_units;
      uint32_t next = 0;
      if (live) next = gridDim.x + static_cast<uint32_t>(atomicAdd(claimed, 1));
      int4 ent = make_int4(-1, 0, 0, 0);
      if (live) {
        const int4 t = __ldg(reinterpret_cast<const int4*>(tiles + u / per_tile));
        ent = make_int4(t.x, t.y, t.z, static_cast<int>(u % per_tile));
      }
      const uint32_t slot = i % kClaimSlots, ph = (i / kClaimSlots) & 1u;
      if (!mbar_wait(&empty[slot], ph ^ 1u, abort_word, lim)) return;
      data[slot] = ent;
      mbar_arrive(&full[slot]);
      if (!live) return;
      u = next;
    }
  }
};

// Last thing a CTA of such a kernel does (one thread, after every role has
// stopped): report a wait that ran out, and let the last CTA of the grid set
// the counters back to zero for the next launch.
__device__ __forceinline__ void finish_claims(int32_t* meta, bool aborted) {
  if (aborted) atomicOr(meta + kWsStatus, kErrTimeout);
  __threadfence();
  if (atomicAdd(meta + kWsFinished, 1) == static_cast<int>(gridDim.x) - 1) {
    atomicExch(meta + kWsClaimed, 0);
    atomicExch(meta + kWsFinished, 0);
  }
}

}  // namespace gmm
