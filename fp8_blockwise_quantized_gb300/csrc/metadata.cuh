// Group metadata on the device: the block-wide pass that fills the workspace,
// and the scan that lets a warp find a call's row tiles from group_sizes alone.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace gmm {

template <typename T>
__device__ __forceinline__ T warp_inclusive_scan(T v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    T o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Exclusive scan over NW warps (thread t of 32 NW); returns the total in
// *total.  warp_sums: NW + 1 entries of shared memory; sync: a barrier of the
// 32 NW threads.
template <int NW, typename Sync>
__device__ __forceinline__ long long block_exclusive_scan(long long v, int t, long long* warp_sums, long long* total,
                                                          Sync&& sync) {
  const int lane = t & 31, warp = t >> 5;
  long long inc = warp_inclusive_scan(v);
  if (lane == 31) warp_sums[warp] = inc;
  sync();
  if (warp == 0) {
    long long w = lane < NW ? warp_sums[lane] : 0;
    long long winc = warp_inclusive_scan(w);
    if (lane < NW) warp_sums[lane] = winc - w;  // exclusive prefix of the warp totals
    if (lane == NW - 1) warp_sums[NW] = winc;
  }
  sync();
  long long r = inc - v + warp_sums[warp];
  *total = warp_sums[NW];
  sync();
  return r;
}

// The metadata of gmm.h's gmm_group_metadata, by 32 NW threads: each owns a
// contiguous run of at most ceil(G / (32 NW)) groups, the block scans the
// per-thread row and tile counts, and every thread then writes its groups'
// offsets, 128-row tiles and 256-row tiles.  keys: G entries of shared memory.
// reset_counters: also zero the work counters (not while a launch that claims
// from them runs).
template <int NW, typename Sync>
__device__ __forceinline__ void write_group_metadata(const int32_t* __restrict__ sizes, int G, int M,
                                                     int32_t* __restrict__ ws, Tile* __restrict__ tiles,
                                                     int32_t* __restrict__ order, Tile* __restrict__ pair_tiles, int t,
                                                     long long* warp_sums, unsigned long long* keys,
                                                     bool reset_counters, Sync&& sync) {
  const int per = (G + 32 * NW - 1) / (32 * NW);
  const int g0 = min(G, t * per), g1 = min(G, g0 + per);

  long long rows = 0, ntiles = 0, npairs = 0;
  constexpr long long kBad = 1LL << 40;  // negative sizes, counted above the pair tiles
  for (int g = g0; g < g1; ++g) {
    const int n = sizes[g];
    if (n < 0) {
      npairs += kBad;
    } else {
      rows += n;
      ntiles += (n + kBM - 1) / kBM;
      npairs += (n + 2 * kBM - 1) / (2 * kBM);
    }
  }
  long long rows_total, tiles_total, pairs_total;
  const long long row_off = block_exclusive_scan<NW>(rows, t, warp_sums, &rows_total, sync);
  const long long tile_off = block_exclusive_scan<NW>(ntiles, t, warp_sums, &tiles_total, sync);
  const long long pair_off = block_exclusive_scan<NW>(npairs, t, warp_sums, &pairs_total, sync);

  int err = 0;
  if (pairs_total >= kBad) err |= kErrNegativeGroup;
  else if (rows_total > M) err |= kErrGroupsExceedM;

  if (err == 0) {
    long long off = row_off, tix = tile_off, pix = pair_off;
    for (int g = g0; g < g1; ++g) {
      const int n = sizes[g];
      ws[kWsOffsets + g] = static_cast<int>(off);
      for (int r = 0; r < n; r += kBM) {
        Tile tl;
        tl.g = g;
        tl.row0 = static_cast<int>(off + r);
        tl.row1 = static_cast<int>(off + min(n, r + kBM));
        tl.pad = 0;
        tiles[tix++] = tl;
      }
      for (int r = 0; r < n; r += 2 * kBM) {
        Tile tl;
        tl.g = g;
        tl.row0 = static_cast<int>(off + r);
        tl.row1 = static_cast<int>(off + min(n, r + 2 * kBM));
        tl.pad = 0;
        pair_tiles[pix++] = tl;
      }
      off += n;
    }
    // the groups by size, descending, ties by index: group g's place is the
    // number of keys (INT32_MAX - size, index) below its own (all keys are
    // distinct), so each thread ranks its groups against all G keys, read as
    // shared-memory broadcasts.  The tgmm kernels deal the units of the
    // largest groups first, so that the last units of the grid are small.
    for (int i = t; i < G; i += 32 * NW)
      keys[i] = (static_cast<unsigned long long>(0x7fffffff - sizes[i]) << 32) | static_cast<unsigned>(i);
    sync();
    for (int i = t; i < G; i += 32 * NW) {
      const unsigned long long mine = keys[i];
      int rank = 0;
      for (int j = 0; j < G; ++j) rank += keys[j] < mine ? 1 : 0;
      order[rank] = i;
    }
  }
  if (t == 0) {
    if (reset_counters) {
      ws[kWsClaimed] = 0;
      ws[kWsFinished] = 0;
    }
    if (err) {
      atomicOr(ws + kWsStatus, err);
      ws[kWsValid] = 0;
      ws[kWsS] = M;
      ws[kWsNumTiles] = 0;
      ws[kWsNumPairTiles] = 0;
    } else {
      ws[kWsValid] = 1;
      ws[kWsS] = static_cast<int>(rows_total);
      ws[kWsNumTiles] = static_cast<int>(tiles_total);
      ws[kWsNumPairTiles] = static_cast<int>(pairs_total);
      ws[kWsOffsets + G] = static_cast<int>(rows_total);
    }
  }
}

// Offsets (G + 1) and the size order (G) of a call with G <= 256 into shared
// memory, by a whole block; keys: G entries of scratch.  Returns whether the
// sizes are valid.  sync: a barrier of the block.
template <typename Sync>
__device__ __forceinline__ bool share_group_order(const int32_t* __restrict__ sizes, int G, int M, int* offsets,
                                                  int* order, unsigned long long* keys, int* valid, Sync&& sync) {
  const int t = threadIdx.x;
  if (t < 32) {
    long long r = 0;
    bool bad = false;
    int n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int g = 8 * t + i;
      n[i] = g < G ? __ldg(sizes + g) : 0;
      bad |= n[i] < 0;
      r += n[i];
    }
    const long long ri = warp_inclusive_scan(r), total = __shfl_sync(0xffffffffu, ri, 31);
    const bool ok = !__any_sync(0xffffffffu, bad) && total <= M;
    int off = static_cast<int>(ri - r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (8 * t + i < G) offsets[8 * t + i] = off;
      off += n[i];
    }
    if (t == 0) {
      *valid = ok ? 1 : 0;
      offsets[G] = static_cast<int>(total);
    }
  }
  // as in write_group_metadata: largest first, ties by index
  if (t < G) keys[t] = (static_cast<unsigned long long>(0x7fffffff - __ldg(sizes + t)) << 32) | static_cast<unsigned>(t);
  sync();
  if (t < G) {
    const unsigned long long mine = keys[t];
    int rank = 0;
    for (int j = 0; j < G; ++j) rank += keys[j] < mine ? 1 : 0;
    order[rank] = t;
  }
  sync();
  return *valid != 0;
}

// Largest G that a kernel takes straight from group_sizes.
constexpr int kScanGroups = 256;

// The row tiles of a call with G <= kScanGroups, in one warp's registers: lane
// l holds groups 8 l .. 8 l + 7.  A kernel that reads group_sizes itself saves
// the metadata launch in front of it (3 us, a quarter of a small call); the
// grid's last CTA fills the workspace meanwhile, for later calls.
struct GroupScan {
  int n[8];
  int off0, tile0;  // rows and row tiles before this lane's groups
  int rows, tiles;  // in all; M and 0 when the sizes are invalid
  __device__ __forceinline__ GroupScan(const int32_t* sizes, int G, int M, int lane) {
    long long r = 0;
    int t = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int g = 8 * lane + i;
      n[i] = g < G ? __ldg(sizes + g) : 0;
      bad |= n[i] < 0;
      r += n[i];
    }
    const long long ri = warp_inclusive_scan(r);
    const long long total = __shfl_sync(0xffffffffu, ri, 31);
    if (__any_sync(0xffffffffu, bad) || total > M) {
      rows = M;
      tiles = off0 = tile0 = 0;
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) t += (n[i] + kBM - 1) / kBM;
    const int ti = warp_inclusive_scan(t);
    rows = static_cast<int>(total);
    tiles = __shfl_sync(0xffffffffu, ti, 31);
    off0 = static_cast<int>(ri - r);
    tile0 = ti - t;
  }
  // Row tile t (the same for all lanes, < tiles): {g, row0, row1, 0}, in every lane.
  __device__ __forceinline__ int4 tile(int t, int lane) const {
    // the last lane whose first tile is at or before t holds it
    const int owner = 31 - __clz(static_cast<int>(__ballot_sync(0xffffffffu, tile0 <= t)));
    int off = off0, left = t - tile0, g = 8 * lane;
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      const int k = (n[i] + kBM - 1) / kBM;
      if (g == 8 * lane + i && left >= k) {
        left -= k;
        off += n[i];
        ++g;
      }
    }
    int size = n[0];
#pragma unroll
    for (int i = 1; i < 8; ++i)
      if (g == 8 * lane + i) size = n[i];
    const int row0 = off + left * kBM, row1 = min(off + size, row0 + kBM);
    return make_int4(__shfl_sync(0xffffffffu, g, owner), __shfl_sync(0xffffffffu, row0, owner),
                     __shfl_sync(0xffffffffu, row1, owner), 0);
  }
};

}  // namespace gmm
