// Work units of the persistent grouped kernels that claim their units as they
// go: a CTA's scheduler warp resolves each unit and hands it to the other
// roles through a queue in shared memory.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "metadata.cuh"
#include "ptx.cuh"

namespace gmm {

constexpr int kClaimSlots = 2;  // entries of a CTA's unit queue

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
  // Scheduler (one warp).  unit(u) gives unit u's row tile and column block
  // (x, y), tile_of(t) row tile t.  A CTA's first kDealt units are dealt round by
  // round (claimed from the start, the CTAs that begin a microsecond early take
  // the units of the others: decoding steps of 264 units ran 23 us instead of
  // 10); the next ones are claimed from the workspace counter, so that a CTA
  // that runs slower takes fewer.  Two claims and the next unit's tile are in
  // flight while a unit is published: a claim and its tile take 1 us or more.
  template <typename U, typename T>
  __device__ void schedule(int* claimed, uint32_t num_units, U&& unit, T&& tile_of, int lane, volatile int* abort_word,
                           uint64_t lim) const {
    constexpr uint32_t kDealt = 4;
    const auto entry = [&](uint32_t u) {
      if (u >= num_units) return make_int4(-1, 0, 0, 0);
      const uint2 at = unit(u);
      int4 t = tile_of(at.x);
      t.w = static_cast<int>(at.y);
      return t;
    };
    uint32_t u = blockIdx.x, u1 = u + gridDim.x, u2 = u1 + gridDim.x;  // u1, u2: lane 0's count
    int4 t = entry(u);
    for (uint32_t i = 0;; ++i) {
      const uint32_t slot = i % kClaimSlots, ph = (i / kClaimSlots) & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], ph ^ 1u, abort_word, lim))) return;
      if (lane == 0) {
        data[slot] = t;
        mbar_arrive(&full[slot]);
      }
      if (u >= num_units) return;
      u = __shfl_sync(0xffffffffu, u1, 0);
      u1 = u2;
      if (lane == 0 && u2 < num_units)
        u2 = i + 3 < kDealt ? u2 + gridDim.x : kDealt * gridDim.x + static_cast<uint32_t>(atomicAdd(claimed, 1));
      t = entry(u);
    }
  }
};

// Runs the scheduler on the call's row tiles: read from group_sizes (sizes not
// NULL), or from the workspace.  make_unit(tiles) returns {number of units, the
// unit map}.
template <typename Args, typename F>
__device__ __forceinline__ void schedule_tiles(const ClaimQueue& queue, const Args& args, F&& make_unit, int lane,
                                               volatile int* abort_word, uint64_t lim) {
  int* claimed = const_cast<int32_t*>(args.meta) + kWsClaimed;
  if (args.sizes) {
    const GroupScan scan(args.sizes, args.G, args.M, lane);
    const auto units = make_unit(static_cast<uint32_t>(scan.tiles));
    queue.schedule(
        claimed, units.num, [&](uint32_t u) { return units.at(u); },
        [&](uint32_t t) { return scan.tile(static_cast<int>(t), lane); }, lane, abort_word, lim);
  } else {
    const auto units = make_unit(static_cast<uint32_t>(args.meta[kWsNumTiles]));
    queue.schedule(
        claimed, units.num, [&](uint32_t u) { return units.at(u); },
        [&](uint32_t t) { return __ldg(reinterpret_cast<const int4*>(args.tiles + t)); }, lane, abort_word, lim);
  }
}

// The epilogue warps' first step (256 threads, tid 0..255): S, the rows that
// belong to a group (every lane); with group_sizes given, the grid's last CTA
// also fills the workspace for later calls.  scratch: 4 KB of shared memory.
template <typename Args>
__device__ __forceinline__ int grouped_rows(const Args& args, int tid, uint8_t* scratch) {
  if (!args.sizes) return args.meta[kWsS];
  if (blockIdx.x == gridDim.x - 1) {
    char* ws = reinterpret_cast<char*>(const_cast<int32_t*>(args.meta));
    const auto sync = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    write_group_metadata<8>(args.sizes, args.G, args.M, const_cast<int32_t*>(args.meta),
                            const_cast<Tile*>(args.tiles),
                            reinterpret_cast<int32_t*>(ws + order_offset_bytes(args.G, args.M)),
                            reinterpret_cast<Tile*>(ws + pair_tiles_offset_bytes(args.G, args.M)), tid,
                            reinterpret_cast<long long*>(scratch),
                            reinterpret_cast<unsigned long long*>(scratch + 128), false, sync);
    sync();  // the scratch is free again
  }
  return GroupScan(args.sizes, args.G, args.M, tid & 31).rows;
}

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
