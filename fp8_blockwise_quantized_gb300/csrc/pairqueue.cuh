// Unit scheduling of the CTA-pair weight-gradient kernels: the unit queue of
// each CTA of a pair and the scheduler that fills both.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace gmm {

constexpr int kChunk = 64;   // rows of the reduction per stage
constexpr int kQueue = 16;   // entries of a CTA's unit queue

// Entry i of a CTA's unit queue (every lane of the calling warp, or the one
// thread of a single-thread role, with `warp_wide` false); the entry is freed
// on the even CTA as soon as it has been read.
struct PairQueue {
  uint64_t* full;
  uint64_t* empty;
  int4* data;
  uint32_t empty_leader;  // shared::cluster address of the even CTA's empty[0]
  bool leader;
  __device__ bool get(uint32_t i, int4& e, bool warp_wide, int lane, volatile int* abort_word,
                      uint64_t lim) const {
    const uint32_t slot = i % kQueue, ph = (i / kQueue) & 1u;
    bool ok = mbar_wait(&full[slot], ph, abort_word, lim);
    if (warp_wide) ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    e = data[slot];
    if (warp_wide) __syncwarp();
    if (lane == 0) {
      if (leader)
        mbar_arrive(&empty[slot]);
      else
        mbar_arrive_remote(empty_leader + slot * 8u);
    }
    return true;
  }
};

// The pair's scheduler: one thread of the even CTA.  taken, ctaken: queue
// entries and chunks that the even CTA's producer has taken.  With splits > 1 a
// group's rows are cut into that many parts of whole chunks: unit u % per_group
// counts them fastest, and its entry holds the part's rows (none where the
// group has too few).
// order and offsets are read with ld (global memory: __ldg).
struct LoadGlobal {
  __device__ __forceinline__ int operator()(const int* p) const { return __ldg(p); }
};
template <typename Load = LoadGlobal>
__device__ __forceinline__ void pair_schedule(const PairQueue& queue, volatile int* taken, volatile int* ctaken,
                                              int* claimed, const int* order, const int* offsets, int G,
                                              int per_group, int num_units, int claim_ahead, int max_batch,
                                              volatile int* abort_word, uint64_t lim, int splits = 1,
                                              Load ld = Load{}) {
  const uint32_t odd_full = mapa_shared(smem_u32(queue.full), 1);
  const uint32_t odd_data = mapa_shared(smem_u32(queue.data), 1);
  uint32_t i = 0;
  auto publish = [&](int4 v) -> bool {
    const uint32_t slot = i % kQueue, ph = (i / kQueue) & 1u;
    // no more than claim_ahead entries beyond the producer (bounded wait)
    if (*taken + claim_ahead <= static_cast<int>(i)) {
      const uint64_t t0 = global_timer_ns();
      while (*taken + claim_ahead <= static_cast<int>(i)) {
        if (*abort_word) return false;
        if (global_timer_ns() - t0 > lim) {
          *abort_word = 1;
          return false;
        }
        __nanosleep(64);
      }
    }
    if (!mbar_wait(&queue.empty[slot], ph ^ 1u, abort_word, lim)) return false;
    queue.data[slot] = v;
    fence_proxy_async_smem();  // the bulk copy reads the entry through the async proxy
    mbar_arrive_expect_tx_remote(odd_full + slot * 8u, 16);
    bulk_copy_s2cluster(odd_data + slot * 16u, &queue.data[slot], 16, odd_full + slot * 8u);
    mbar_arrive(&queue.full[slot]);
    ++i;
    return true;
  };
  constexpr int kMaxBatch = 4;
  // Claim q takes unit q/2 from the large end of the size order when q is
  // even and unit num_units-1-q/2 from the small end when q is odd, so every
  // pair alternates long, read-heavy units with short ones whose cost is
  // mostly the dW store (or only that, for an empty group): the loads of the
  // one overlap the stores of the other, and the launch never runs a phase of
  // loads only followed by a phase of stores only.
  // With groups of about one size there is nothing to mix, and the plain
  // order keeps each group's units together: alternate only when the
  // largest group has more than twice the chunks of the smallest.
  bool mix = false;
  if (num_units > 0) {
    const int gl = ld(order), gs = ld(order + G - 1);
    const int cl = (ld(offsets + gl + 1) - ld(offsets + gl) + kChunk - 1) / kChunk;
    const int cs = (ld(offsets + gs + 1) - ld(offsets + gs) + kChunk - 1) / kChunk;
    mix = cl > 2 * cs;
  }
  auto unit_of = [&](int q) { return (mix && (q & 1)) ? num_units - 1 - (q >> 1) : (mix ? (q >> 1) : q); };
  // Claims are paced by work: the next claim is made only once the producer
  // is within kLeadChunks chunks of the end of what is already published, so
  // that a claimed unit starts within a few microseconds (the units of one
  // group, claimed one after the other, then read its rows at about the same
  // time and find them in L2, instead of one of them waiting behind a long
  // unit and reading them again after they were evicted).
  constexpr int kLeadChunks = 8;
  bool ok = true;
  int batch = min(mix ? 2 : 1, max_batch);
  int published = 0;  // chunks of the published units (1 for an empty group's)
  while (ok) {
    if (published - *ctaken >= kLeadChunks) {
      const uint64_t t0 = global_timer_ns();
      while (published - *ctaken >= kLeadChunks) {
        if (*abort_word || global_timer_ns() - t0 > lim) break;
        __nanosleep(64);
      }
      if (*abort_word || published - *ctaken >= kLeadChunks) {
        *abort_word = 1;
        ok = false;
        break;
      }
    }
    const int k0 = atomicAdd(claimed, batch);
    if (k0 >= num_units) break;
    const int cnt = min(batch, num_units - k0);
    int u[kMaxBatch], g[kMaxBatch], r0[kMaxBatch], r1[kMaxBatch];
#pragma unroll
    for (int j = 0; j < kMaxBatch; ++j) u[j] = j < cnt ? unit_of(k0 + j) : 0;
#pragma unroll
    for (int j = 0; j < kMaxBatch; ++j) g[j] = j < cnt ? ld(order + u[j] / per_group) : 0;
#pragma unroll
    for (int j = 0; j < kMaxBatch; ++j) {
      r0[j] = j < cnt ? ld(offsets + g[j]) : 0;
      r1[j] = j < cnt ? ld(offsets + g[j] + 1) : 0;
      if (splits > 1) {
        const int part = ((r1[j] - r0[j] + kChunk - 1) / kChunk + splits - 1) / splits * kChunk;
        r0[j] = min(r1[j], r0[j] + part * (u[j] % per_group % splits));
        r1[j] = min(r1[j], r0[j] + part);
      }
    }
#pragma unroll
    for (int j = 0; j < kMaxBatch; ++j) {
      if (ok && j < cnt) {
        ok = publish(make_int4(g[j], u[j] % per_group, r0[j], r1[j]));
        published += max(1, (r1[j] - r0[j] + kChunk - 1) / kChunk);
      }
    }
    // the large-end units shrink as the claims go on: claim more at once
    // when they get small (when mixing, the first claim of the batch is a
    // large-end one whenever the batch size is even)
    const int jf = (mix && (k0 & 1)) ? (cnt > 1 ? 1 : 0) : 0;
    const int chunks = (r1[jf] - r0[jf] + kChunk - 1) / kChunk;
    batch = min(chunks >= 4 ? (mix ? 2 : 1) : chunks >= 2 ? 2 : 4, max_batch);
  }
  if (ok) publish(make_int4(-1, 0, 0, 0));
}

}  // namespace gmm
