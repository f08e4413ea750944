// The expert weight gradient from an 8-bit activation checkpoint:
//   dW[g][k, n] = sum over the rows m of group g of  xq[m, k] xs[k/128, m] dy[m, n]
// with xq e4m3 codes in 1x128 blocks and fp32 scales (as gmm_quantize_lhs
// writes them), dy bf16, fp32 accumulation, bf16 output; an empty group gets 0.
//
// The tensor core takes both operands of one product in one type, and the
// scale runs along the reduction (one per row and 128 columns), so it cannot
// be applied to the sums: the codes are expanded to bf16, scaled, on their way
// from shared memory to shared memory.  Scaling rounds each value once to bf16
// (at most 2^-8 of it, against the 2^-4 of the e4m3 code it expands; the result
// is 0.0018 off in norm, 0.0017 of which its own rounding to bf16 makes).  In
// exchange x is read at one byte an element.
//
// A cluster of two CTAs on the two SMs of a pair owns the tile (g, 256 rows of
// K, 256 columns of N) and walks the group's rows in chunks of 64; each CTA
// holds 128 k columns and 128 n columns (608 threads):
//   warp 0       TMA: the chunk's codes (64 x 128 bytes) and dy (two 64 x 64
//                boxes) into a ring of kRing slots
//   warps 11-18  expand the codes to bf16 (MN-major 128-byte swizzled boxes)
//                into one of kOper operand buffers, two groups of four warps
//                taking every other chunk; rows past the group's end become
//                zeros there, and in dy, whatever the rows of the next group
//                hold
//   warp 1       even CTA: one M=256 tcgen05.mma (cta_group::2) per 16 rows
//                over both CTAs' shared memory
//   warps 2-9    epilogue: 128 k rows x 256 columns per CTA, as bf16 boxes
//   warp 10      even CTA: the pair's scheduler
// Tiles that reach past K or N (multiples of 128) load zeros and store nothing
// there.
//
// 310 us at the production gate/up layer (256 experts, 65536 rows, K 2048, N
// 1024, Zipf routing), 4.3 TB/s: HBM under a mix of one byte read to 3.4
// written, for which 4.6 to 5.0 TB/s are reached at best here; without the
// expansion 285, without the stores 275.  One group of expanding warps instead
// of two: 391.
//
// Few tiles and many rows (one group of 65536 rows, K = N = 256: one tile) would
// leave most pairs idle: then each group's rows are cut into `splits` parts whose
// fp32 sums go to a scratch tensor, and a second kernel adds them in order (the
// same bits every time) and rounds once.
#include "common.cuh"
#include "kernels.cuh"
#include "metadata.cuh"
#include "pairqueue.cuh"
#include "ptx.cuh"
#include "unitqueue.cuh"

namespace gmm {

namespace {

constexpr int BN = 256;
constexpr int kThreads = 608;
constexpr int kEpiWarps = 8;
constexpr int kSchedWarp = 10;
constexpr int kExpandWarp0 = 11;
constexpr int kExpandWarps = 4;  // per group
constexpr int kGroups = 2;
constexpr int kRing = 5;
constexpr int kOper = 4;
constexpr uint64_t kDrainLimitNs = 200000000ull;
// producer, epilogue and expanding warps of both CTAs, and the MMA issuer
constexpr int kReaders = 2 * (1 + kEpiWarps + kGroups * kExpandWarps) + 1;

constexpr int kBoxBytes = kChunk * 128;      // 64 rows x 128 bytes
constexpr int kSlotBytes = 3 * kBoxBytes;    // codes, two boxes of dy
constexpr int kOperBytes = 2 * kBoxBytes;    // 64 rows x 128 bf16
constexpr int kStagingBytes = kEpiWarps * 4096;
constexpr int kBarBytes = 1024;
constexpr int kGroupBytes = 4 * (2 * kScanGroups + 4);  // offsets and order of a call that scans its sizes
constexpr int kSmemBytes = 1024 + kRing * kSlotBytes + kOper * kOperBytes + kStagingBytes + kBarBytes + kGroupBytes;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
static_assert(16 * kQueue + 8 * (2 * kRing + kOper + 5 + 2 * kQueue) + 16 <= kBarBytes, "barrier area");

// 4 e4m3 codes times a scale, as two packed bf16 pairs
__device__ __forceinline__ uint2 expand4(uint32_t codes, float scale) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes >> 16), __NV_E4M3);
  const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
  return make_uint2(pack_bf16x2(a.x * scale, a.y * scale), pack_bf16x2(b.x * scale, b.y * scale));
}

// SPLIT: the parts' fp32 sums to the scratch tensor [splits * G * K, N] that
// map_dw describes (32 x 32 boxes) instead of bf16 dw (64 x 32 boxes).
template <bool SPLIT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    tgmm_ckpt_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_dy,
                     const __grid_constant__ CUtensorMap map_dw, const TgmmArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* oper = ring + kRing * kSlotBytes;
  uint8_t* staging = oper + kOper * kOperBytes;
  int4* qdata = reinterpret_cast<int4*>(staging + kStagingBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(qdata + kQueue);  // each CTA: its slot has landed
  uint64_t* empty = full + kRing;    // each CTA: the pair's products of the chunk in the slot are done
  uint64_t* ready = empty + kRing;   // even CTA: both CTAs have expanded the chunk
  uint64_t* tfull = ready + kOper;
  uint64_t* tempty = tfull + 2;      // even CTA: both CTAs' epilogues freed the accumulator
  uint64_t* drain = tempty + 2;
  uint64_t* qfull = drain + 1;
  uint64_t* qempty = qfull + kQueue;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(qempty + kQueue);
  volatile int* abort_word = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* taken = abort_word + 1;
  volatile int* ctaken = taken + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    *taken = 0;
    *ctaken = 0;
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int j = 0; j < kOper; ++j) mbar_init(&ready[j], 2 * kExpandWarps);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    for (int q = 0; q < kQueue; ++q) {
      mbar_init(&qfull[q], 1);
      mbar_init(&qempty[q], kReaders);
    }
    *abort_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_dy);
    tma_prefetch_desc(&map_dw);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are initialised before any remote arrive
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  griddep_launch_dependents();
  griddep_wait();  // inputs, metadata and the work counter come from earlier kernels

  const int KT = (args.K + 255) / 256, NT = (args.N + BN - 1) / BN;
  const int splits = SPLIT ? args.splits : 1;
  const int per_group = KT * NT * splits;
  // group offsets and size order: from the workspace, or of group_sizes in
  // shared memory (the scheduler's CTA alone needs them)
  int* shared_offsets = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(qdata) + kBarBytes);
  int* shared_order = shared_offsets + kScanGroups + 1;
  bool valid;
  if (args.sizes) {
    valid = leader && share_group_order(args.sizes, args.G, args.M, shared_offsets, shared_order,
                                        reinterpret_cast<unsigned long long*>(staging), shared_order + kScanGroups,
                                        [] { __syncthreads(); });
  } else {
    valid = args.meta[kWsValid] != 0;
  }
  const int num_units = valid ? args.G * per_group : 0;
  const uint64_t lim = args.wait_limit_ns;
  const PairQueue queue{qfull, qempty, qdata, mapa_shared(smem_u32(qempty), 0), leader};

  if (warp == 0) {
    if (lane == 0) {
      uint32_t c = 0;
      bool ok = true;
      int4 e;
      int issued = 0;
      for (uint32_t i = 0; ok && queue.get(i, e, false, 0, abort_word, lim) && e.x >= 0; ++i) {
        *taken = static_cast<int>(i) + 1;
        if (e.w <= e.z) *ctaken = ++issued;  // an empty group's unit counts as one chunk
        const int k0 = (e.y / splits / NT) * 256 + static_cast<int>(rank) * 128;
        const int n0 = (e.y / splits % NT) * BN + static_cast<int>(rank) * 128;
        for (int r = e.z; r < e.w; r += kChunk) {
          const uint32_t s = c % kRing, ph = (c / kRing) & 1u;
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_word, lim)) {
            ok = false;
            break;
          }
          uint8_t* slot = ring + s * kSlotBytes;
          mbar_arrive_expect_tx(&full[s], kSlotBytes);
          tma_load_2d(slot, &map_x, &full[s], k0, r);
          tma_load_2d(slot + kBoxBytes, &map_dy, &full[s], n0, r);
          tma_load_2d(slot + 2 * kBoxBytes, &map_dy, &full[s], n0 + 64, r);
          ++c;
          *ctaken = ++issued;
        }
      }
      // wait for the last copy issued into every slot (they land in microseconds)
      volatile int no_abort = 0;
      for (uint32_t s = 0; s < kRing; ++s) {
        if (c > s) {
          const uint32_t last = s + kRing * ((c - 1 - s) / kRing);
          mbar_wait(&full[s], (last / kRing) & 1u, &no_abort, kDrainLimitNs);
        }
      }
    }
  } else if (warp == 1) {
    if (leader && lane == 0) {
      constexpr uint32_t idesc = make_idesc(1u /*bf16*/, true, true, 2 * kBM, BN);
      const uint32_t a_lo0 = desc_lo_sw128(smem_u32(oper), kBoxBytes);
      const uint32_t b_lo0 = desc_lo_sw128(smem_u32(ring) + kBoxBytes, kBoxBytes);
      RingPos<kRing> r;
      RingPos<kOper> o;
      RingPos<2> acc;
      bool ok = true, any = false, next_ready = false;
      int4 e;
      for (uint32_t i = 0; ok && queue.get(i, e, false, 0, abort_word, lim) && e.x >= 0; ++i) {
        if (e.w <= e.z) continue;  // empty group: the epilogues write zeros
        if (!mbar_wait(&tempty[acc.slot], acc.phase ^ 1u, abort_word, lim)) break;
        tc_fence_after();
        const uint32_t d = tbase + acc.slot * BN;
        uint32_t more = 0;  // the unit's first product overwrites the accumulator
        for (int live = e.w - e.z; live > 0; live -= kChunk) {
          if (!next_ready && !mbar_wait(&ready[o.slot], o.phase, abort_word, lim)) {
            ok = false;
            break;
          }
          const uint32_t a_lo = a_lo0 + o.slot * (kOperBytes >> 4), b_lo = b_lo0 + r.slot * (kSlotBytes >> 4);
          uint64_t* freed = &empty[r.slot];
          r.advance();
          o.advance();
          next_ready = mbar_test(&ready[o.slot], o.phase);  // answered while the products are issued
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (16 * q < live)
              mma_bf16_pair(d, desc_sw128(a_lo + (2048 >> 4) * q), desc_sw128(b_lo + (2048 >> 4) * q), idesc,
                            q > 0 ? 1u : more);
          }
          mma_commit_pair(freed, 0x3);
          more = 1;
        }
        any |= more != 0;
        if (!ok) break;
        mma_commit_pair(&tfull[acc.slot], 0x3);
        acc.advance();
      }
      if (any) {
        volatile int no_abort = 0;
        mma_commit_pair(drain, 0x1);
        mbar_wait(drain, 0, &no_abort, kDrainLimitNs);
      }
    }
  } else if (warp < 2 + kEpiWarps) {
    grouped_rows(args, static_cast<int>(threadIdx.x) - 64, staging);
    const int pw = warp - 2;
    const int half = pw >> 2;
    const int quad = warp & 3;
    const uint32_t t_lane = tbase + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
    uint8_t* box = staging + pw * 4096;
    uint8_t* brow = box + lane * 128;
    uint32_t t = 0;
    int4 e;
    for (uint32_t i = 0; queue.get(i, e, true, lane, abort_word, lim) && e.x >= 0; ++i) {
      const int k0 = (e.y / splits / NT) * 256 + static_cast<int>(rank) * 128;
      const int n0 = (e.y / splits % NT) * BN + half * 128;
      const bool inside = k0 < args.K && n0 < args.N;
      const int y = (SPLIT ? e.y % splits * args.G + e.x : e.x) * args.K + k0 + quad * 32;
      const bool some = e.w > e.z;
      const uint32_t b = t & 1u;
      if (some) {
        if (!__all_sync(0xffffffffu, mbar_wait(&tfull[b], (t >> 1) & 1u, abort_word, lim))) break;
        tc_fence_after();
        ++t;
      }
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        uint32_t r[64];
        if (some) {
          const uint32_t ta = t_lane + b * BN + half * 128 + 64 * pass;
          tmem_ld_32x32(ta, *reinterpret_cast<uint32_t(*)[32]>(r));
          tmem_ld_32x32(ta + 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
          tmem_ld_wait();
          if (pass == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(tempty0 + b * 8u);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 64; ++j) r[j] = 0u;
        }
        if (!inside) continue;
        if (SPLIT) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (lane == 0) bulk_wait_read_all();  // the previous store has read the box
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int c = 32 * q + 4 * j;
              *reinterpret_cast<uint4*>(brow + ((j ^ (lane & 7)) << 4)) = make_uint4(r[c], r[c + 1], r[c + 2], r[c + 3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&map_dw, box, n0 + 64 * pass + 32 * q, y);
              bulk_commit();
            }
          }
          continue;
        }
        if (lane == 0) bulk_wait_read_all();  // the previous store has read the box
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = 8 * j;
          *reinterpret_cast<uint4*>(brow + ((j ^ (lane & 7)) << 4)) =
              make_uint4(pack_bf16x2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])),
                         pack_bf16x2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])),
                         pack_bf16x2(__uint_as_float(r[c + 4]), __uint_as_float(r[c + 5])),
                         pack_bf16x2(__uint_as_float(r[c + 6]), __uint_as_float(r[c + 7])));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&map_dw, box, n0 + 64 * pass, y);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  } else if (warp == kSchedWarp) {
    if (leader && lane == 0) {
      int* claimed = const_cast<int32_t*>(args.meta) + kWsClaimed;
      if (args.sizes)
        pair_schedule(queue, taken, ctaken, claimed, shared_order, shared_offsets, args.G, per_group, num_units, 3, 4,
                      abort_word, lim, splits, [](const int* p) { return *p; });
      else
        pair_schedule(queue, taken, ctaken, claimed, args.order, args.meta + kWsOffsets, args.G, per_group, num_units,
                      3, 4, abort_word, lim, splits);
    }
  } else if (warp >= kExpandWarp0) {
    // thread: row `row` of the chunk, 64 of its 128 codes (half `hb`)
    const int et = static_cast<int>(threadIdx.x) - 32 * kExpandWarp0;
    const uint32_t group = static_cast<uint32_t>(et) / (32 * kExpandWarps);
    const int row = et % (32 * kExpandWarps) >> 1, hb = et & 1;
    const uint32_t ready0 = mapa_shared(smem_u32(ready), 0);
    static_assert(kGroups == 2 && kOper == kRing - 1, "the positions below");
    RingPos<kRing> s;      // the chunk's slot
    RingPos<kOper> o;      // its operand buffer
    // That buffer is free once the products of the chunk kOper before are done:
    // it lay in the slot after this one (kRing - kOper on).  That slot's next
    // phase cannot complete before this chunk's, so the parity is unambiguous.
    uint32_t c = 0;        // chunks so far
    bool ok = true;
    int4 e;
    for (uint32_t i = 0; ok && queue.get(i, e, true, lane, abort_word, lim) && e.x >= 0; ++i) {
      const int k0 = (e.y / splits / NT) * 256 + static_cast<int>(rank) * 128;
      const float* xs = args.xs + static_cast<long long>(k0 / 128) * args.M;
      const bool inside = k0 < args.K;
      // this group's chunks of the unit; a chunk's scale is loaded one ahead
      const int mine = ((c & 1) == group ? 0 : kChunk) + row;
      float next = inside && e.z + mine < e.w ? __ldg(xs + e.z + mine) : 0.0f;
      for (int r = e.z; r < e.w; r += kChunk, ++c, s.advance(), o.advance()) {
        if ((c & 1) != group) continue;
        const float scale = next;
        const int ahead = r + kGroups * kChunk + row;
        next = inside && ahead < e.w ? __ldg(xs + ahead) : 0.0f;
        const int live = e.w - r;
        bool got = mbar_wait(&full[s.slot], s.phase, abort_word, lim);
        if (got && c >= kOper) {
          RingPos<kRing> f = s;
          f.advance();  // kOper chunks back: the next slot, in the phase before
          got = mbar_wait(&empty[f.slot], f.phase ^ 1u, abort_word, lim);
        }
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        uint8_t* slot = ring + s.slot * kSlotBytes;
        const uint8_t* src = slot + row * 128;
        uint8_t* dst = oper + o.slot * kOperBytes + hb * kBoxBytes + row * 128;
        const int sw = row & 7;
        if (row < live) {
          // 16 codes at a time; the halves run in opposite order so that their
          // stores fall into different banks
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int ch = q ^ (hb << 1);
            const uint4 v = *reinterpret_cast<const uint4*>(src + (((4 * hb + ch) ^ sw) << 4));
            const uint2 a = expand4(v.x, scale), b = expand4(v.y, scale);
            const uint2 d = expand4(v.z, scale), f = expand4(v.w, scale);
            *reinterpret_cast<uint4*>(dst + (((2 * ch) ^ sw) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
            *reinterpret_cast<uint4*>(dst + (((2 * ch + 1) ^ sw) << 4)) = make_uint4(d.x, d.y, f.x, f.y);
          }
        } else if (row < ((live + 15) & ~15)) {
          // the 16-row step that crosses the group's end: zeros on both sides
          uint8_t* dyrow = slot + (1 + hb) * kBoxBytes + row * 128;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            *reinterpret_cast<uint4*>(dst + 16 * q) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(dyrow + 16 * q) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();  // the tensor core reads what was written here
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(ready0 + o.slot * 8u);
      }
    }
  }

  // teardown: no CTA of the pair leaves while the other may still arrive on
  // its barriers or its products may still touch the other's TMEM
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, 2 * BN);
  }
  if (threadIdx.x == 0) {
    int32_t* w = const_cast<int32_t*>(args.meta);
    if (*abort_word) atomicOr(w + kWsStatus, kErrTimeout);
    // every CTA has stopped claiming; the last one out resets the counters
    __threadfence();
    if (atomicAdd(w + kWsFinished, 1) == static_cast<int>(gridDim.x) - 1) {
      atomicExch(w + kWsClaimed, 0);
      atomicExch(w + kWsFinished, 0);
    }
  }
}

// dw = bf16(sum over the parts, in order), four elements a thread.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float4* __restrict__ parts, long long n4, int splits,
                                                        uint2* __restrict__ dw) {
  griddep_launch_dependents();
  griddep_wait();
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n4;
       i += static_cast<long long>(gridDim.x) * 256) {
    float4 a = __ldg(parts + i);
    for (int s = 1; s < splits; ++s) {
      const float4 b = __ldg(parts + s * n4 + i);
      a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
    }
    dw[i] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
}

template <bool SPLIT>
cudaError_t launch(const CUtensorMap& map_x, const CUtensorMap& map_dy, const CUtensorMap& map_dw,
                   const TgmmArgs& args, int max_pairs, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  static std::atomic<int> resident[64];
  auto kernel = tgmm_ckpt_kernel<SPLIT>;
  cudaError_t e = allow_smem(kernel, kSmemBytes, done);
  int dev = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // as many pairs as can be resident at once (one CTA per SM), asked once per device
  int clusters = resident[dev & 63].load(std::memory_order_relaxed);
  if (clusters == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * 1024, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    resident[dev & 63].store(clusters, std::memory_order_relaxed);
  }
  const int pairs = clusters < max_pairs ? clusters : max_pairs;
  return launch_pdl(kernel, dim3(2 * pairs), dim3(kThreads), kSmemBytes, stream, map_x, map_dy, map_dw, args);
}

}  // namespace

// The fewest parts that bring the busiest pair's share of the rows down by a
// tenth or more; no more than two units per pair (the parts' sums are written
// and read again) and at least eight chunks per part of a mean group (one group
// of 65536 rows, K = N = 256: 73 parts, 35 us for 387; 4 groups of 4096, K 1024,
// N 512: 2 parts, 27 us for 33; 16 groups of 1250, K 512, N 256 in 2 parts of
// ten chunks: 18 us for 16).
int tgmm_ckpt_splits(int G, int64_t M, int64_t K, int64_t N, int sms) {
  const int64_t units = static_cast<int64_t>(G) * ((K + 255) / 256) * ((N + BN - 1) / BN), pairs = sms / 2;
  int best = 1;
  double share = static_cast<double>((units + pairs - 1) / pairs);
  for (int s = 2; s * units <= 2 * pairs && s <= M / (8LL * kChunk * G); ++s) {
    const double v = static_cast<double>((s * units + pairs - 1) / pairs) / s;
    if (v < 0.9 * share) best = s, share = v;
  }
  return best;
}

cudaError_t launch_tgmm_ckpt(const CUtensorMap& map_x, const CUtensorMap& map_dy, const CUtensorMap& map_dw,
                             const TgmmArgs& args, int max_pairs, cudaStream_t stream) {
  if (args.splits <= 1) return launch<false>(map_x, map_dy, map_dw, args, max_pairs, stream);
  cudaError_t e = launch<true>(map_x, map_dy, map_dw, args, max_pairs, stream);
  if (e != cudaSuccess) return e;
  const long long n4 = static_cast<long long>(args.G) * args.K * args.N / 4;
  const long long ctas = (n4 + 255) / 256;
  return launch_pdl(sum_parts_kernel, dim3(static_cast<unsigned>(ctas < 4096 ? ctas : 4096)), dim3(256), 0, stream,
                    reinterpret_cast<const float4*>(args.parts), n4, args.splits, reinterpret_cast<uint2*>(args.dw));
}

}  // namespace gmm
