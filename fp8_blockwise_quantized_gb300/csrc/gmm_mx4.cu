// MXFP4 grouped GEMM: out[m, n] = bf16( sum over blocks of 32 along K of
//   2^(sx - 127) 2^(sw - 127) sum_k cx[m, k] cw[g, n, k] ),  m in group g,
// on the block-scaled tensor core (kind::mxf4: packed E2M1 operands, E8M0
// scales applied in the product, fp32 sums).  With a gate | up weight the
// output is silu(gate) * up, as bf16 and / or as MXFP4 for the next product.
//
// 512 threads, one persistent CTA per SM, units of 128 rows x BN weight columns:
//   warp 0       TMA: per K step of 256 (128 packed bytes a row) the codes of
//                128 rows and of BN columns into a ring slot
//   warp 1       tcgen05.mma, K = 64, four per K step
//   warp 2       claims the CTA's units and queues them for the other roles
//   warps 4-11   epilogue
//   warps 12-15  scales: lane l holds the scale words (four blocks of 32) of
//                rows l, l + 32, l + 64, l + 96, which is the layout the tensor
//                core reads, once in every lane quarter of the tensor memory.
//                Each warp stores one quarter, straight from registers.
//                (Copies from shared memory, tcgen05.cp, run in the MMAs' pipe
//                and stopped them 60 cycles each: 117 instead of 99 us for the
//                gate/up product of 65536 rows, 256 experts, K 2048, N 512.)
// That product takes 94 us now (4.4 TB/s, 2.9 PFLOP/s; floor 61 us of HBM): a
// quarter of it are unit boundaries, the rest waits for operands.  The second
// one of that layer (K 512, N 2048) takes 76 us, 5.6 TB/s, two thirds writes.
// BN = 256 fills half of the tensor memory with one accumulator and needs the
// rest for the scales, so the epilogue's loads stop the products of the next
// unit (its operands are fetched meanwhile); BN = 128 has two accumulators.
#include "common.cuh"
#include "kernels.cuh"
#include "mx4.cuh"
#include "ptx.cuh"
#include "rowbox.cuh"
#include "unitqueue.cuh"

namespace gmm {

namespace {

constexpr int kThreads = 512;
constexpr int kEpiWarps = 8;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kScaleWarp0 = 12;
constexpr int kScaleWarps = 4;
constexpr int kQueueReaders = 2 + kEpiWarps + kScaleWarps;
constexpr uint64_t kDrainLimitNs = 200000000ull;
// The scales come in slots of kScaleBlocks 128-wide K blocks (four K steps): a
// slot costs its loads' latency and a store to tensor memory, whatever its size
// (two steps a slot: 99 us for 94 in the gate/up product named above).
constexpr int kScaleBlocks = 8;
// Register split: 128 per thread at launch; the epilogue warpgroups take a
// whole 32 x 128 part of the accumulator into registers at once.
constexpr uint32_t kControlRegs = 56, kEpiRegs = 168, kScaleRegs = 120;
static_assert(128 * (kControlRegs + kScaleRegs) + 256 * kEpiRegs <= kThreads * 128,
              "register split exceeds the launch budget");

enum Mx4Mode { kPlain = 0, kFused = 1, kFusedQuant = 2 };

template <int BN, bool FUSE>
struct Mx4Tile {
  static constexpr int kTilesB = BN / 128;             // 128-column scale tiles
  static constexpr int kBoxes = FUSE ? 1 : kTilesB;    // 32 x 64 staging boxes per warp
  static constexpr int kStages = kBoxes == 2 ? 3 : (BN == 256 ? 4 : 5);
  static constexpr int kBufs = BN == 256 ? 1 : 2;
  static constexpr int kABytes = kBM * 128;
  static constexpr int kBBytes = BN * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kScaleCol0 = 256;                               // first tensor-memory column of the scales
  static constexpr int kScaleCols = kScaleBlocks * 4 * (1 + kTilesB);  // columns per scale slot
  static constexpr int kScaleSlots = 256 / kScaleCols;
  static constexpr int kStagingBytes = kEpiWarps * kBoxes * 4096;
  static constexpr int kBarBytes = 512;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kStagingBytes + kBarBytes;
  static_assert(kBufs * BN <= kScaleCol0 && kScaleCol0 + kScaleSlots * kScaleCols <= 512, "tensor memory");
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static_assert(8 * (2 * kStages + 2 * kScaleSlots + 2 * kBufs + 1 + ClaimQueue::kBarriers) + 16 + 16 * kClaimSlots <= kBarBytes,
                "barrier area");
};

// Unit u: row tile u / per_tile, column block u % per_tile.
struct Mx4Units {
  uint32_t num, per_tile;
  __device__ uint2 at(uint32_t u) const { return make_uint2(u / per_tile, u % per_tile); }
};

// Instruction descriptor of kind::mxf4: E2M1 operands (bits 7-9, 10-11: 1),
// E8M0 scales (bit 23), N >> 3 in bits 17-22, M >> 7 in bits 27-28; which pair
// of a scale word's four bytes applies (0 or 2): B's in bits 4-5, A's in 29-30.
template <int BN>
__device__ __forceinline__ uint32_t mx4_idesc(uint32_t pair) {
  return (1u << 7) | (1u << 10) | (1u << 23) | (static_cast<uint32_t>(BN >> 3) << 17) | (1u << 27) | (pair << 4) |
         (pair << 29);
}

template <int BN, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    gmm_mx4_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_out, const Mx4Args args) {
  constexpr bool FUSE = MODE != kPlain;
  using C = Mx4Tile<BN, FUSE>;
  constexpr int kStages = C::kStages, kBufs = C::kBufs, kScaleSlots = C::kScaleSlots;
  constexpr int kOutCols = FUSE ? BN / 2 : BN;
  constexpr int kWarpCols = kOutCols / 2;  // output columns per epilogue warp
  constexpr bool kHalfTiles = FUSE && BN == 128;  // a unit uses 64 columns of two scale tiles of w
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* staging = ring + kStages * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + C::kStagingBytes);
  uint64_t* empty = full + kStages;
  uint64_t* sfull = empty + kStages;
  uint64_t* sempty = sfull + kScaleSlots;
  uint64_t* tfull = sempty + kScaleSlots;
  uint64_t* tempty = tfull + kBufs;
  uint64_t* drain = tempty + kBufs;
  uint64_t* ufull = drain + 1;
  uint64_t* uempty = ufull + kClaimSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(uempty + kClaimSlots);
  volatile int* abort_word = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int4* udata = reinterpret_cast<int4*>((reinterpret_cast<uintptr_t>(tmem_slot + 2) + 15) & ~uintptr_t{15});
  const ClaimQueue queue{ufull, uempty, udata};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int q = 0; q < kScaleSlots; ++q) {
      mbar_init(&sfull[q], kScaleWarps);
      mbar_init(&sempty[q], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps);
    }
    mbar_init(drain, 1);
    queue.init(kQueueReaders);
    *abort_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_b);
    tma_prefetch_desc(&map_out);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  griddep_launch_dependents();
  griddep_wait();  // inputs and metadata come from earlier kernels

  const int KB = args.K / 128, KS = (KB + 1) / 2;
  const int Nw = FUSE ? 2 * args.N : args.N;
  const uint64_t lim = args.wait_limit_ns;

  if (warp < kEpiWarp0) regs_dec<kControlRegs>();
  if (warp == 0) {
    if (lane == 0) {
      RingPos<kStages> r;
      uint32_t c = 0;
      bool ok = true;
      int4 e;
      for (uint32_t i = 0; ok && queue.get(i, e, false, 0, abort_word, lim) && e.x >= 0; ++i) {
        const int brow = e.x * Nw + e.w * kOutCols;
        for (int ks = 0; ks < KS; ++ks) {
          if (!mbar_wait(&empty[r.slot], r.phase ^ 1u, abort_word, lim)) {
            ok = false;
            break;
          }
          uint8_t* dst = ring + r.slot * C::kStageBytes;
          uint64_t* bar = &full[r.slot];
          mbar_arrive_expect_tx(bar, C::kStageBytes);
          // past K (an odd number of 128-wide blocks) the copies bring zeros
          tma_load_2d(dst, &map_a, bar, ks * 128, e.y);
          tma_load_2d(dst + C::kABytes, &map_b, bar, ks * 128, brow);
          if (FUSE) tma_load_2d(dst + C::kABytes + C::kBBytes / 2, &map_b, bar, ks * 128, brow + args.N);
          r.advance();
          ++c;
        }
      }
      // wait for the last copy issued into every slot (they land in microseconds)
      volatile int no_abort = 0;
      for (uint32_t s = 0; s < kStages; ++s) {
        if (c > s) {
          const uint32_t last = s + kStages * ((c - 1 - s) / kStages);
          mbar_wait(&full[s], (last / kStages) & 1u, &no_abort, kDrainLimitNs);
        }
      }
    }
  } else if (warp == 1) {
    // The tensor core's queue is short: whatever this thread does between two
    // steps' products beyond some 200 cycles is time without products, so the
    // loop keeps running positions and descriptor words instead of deriving them.
    if (lane == 0) {
      const uint32_t ring_lo = desc_lo_sw128(smem_u32(ring), 16);
      const uint32_t tsc = tbase + C::kScaleCol0;
      RingPos<kStages> r;
      RingPos<kScaleSlots> q;
      RingPos<kBufs> acc;
      bool ok = true, any = false, next_ready = false;
      int4 e;
      for (uint32_t i = 0; ok && queue.get(i, e, false, 0, abort_word, lim) && e.x >= 0; ++i) {
        if (!mbar_wait(&tempty[acc.slot], acc.phase ^ 1u, abort_word, lim)) break;
        const uint32_t d = tbase + acc.slot * BN;
        uint32_t more = 0;  // the unit's first product overwrites the accumulator
        for (int kb = 0; kb < KB; kb += kScaleBlocks) {
          if (!mbar_wait(&sfull[q.slot], q.phase, abort_word, lim)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // the slot's scale columns: x's K blocks (4 columns each), then w's
          uint32_t tsa = tsc + q.slot * C::kScaleCols, tsb = tsa + 4 * kScaleBlocks;
#pragma unroll
          for (int step = 0; step < kScaleBlocks / 2; ++step) {
            if (kb + 2 * step >= KB) break;
            if (!next_ready && !mbar_wait(&full[r.slot], r.phase, abort_word, lim)) {
              ok = false;
              break;
            }
            const uint32_t a_lo = ring_lo + r.slot * (C::kStageBytes >> 4), b_lo = a_lo + (C::kABytes >> 4);
            uint64_t* freed = &empty[r.slot];
            r.advance();
            next_ready = mbar_test(&full[r.slot], r.phase);  // answered while the products are issued
            mma_mx4(d, desc_sw128(a_lo), desc_sw128(b_lo), mx4_idesc<BN>(0), tsa, tsb, more);
            mma_mx4(d, desc_sw128(a_lo + 2), desc_sw128(b_lo + 2), mx4_idesc<BN>(2), tsa, tsb, 1);
            if (kb + 2 * step + 1 < KB) {
              tsa += 4, tsb += 4 * C::kTilesB;
              mma_mx4(d, desc_sw128(a_lo + 4), desc_sw128(b_lo + 4), mx4_idesc<BN>(0), tsa, tsb, 1);
              mma_mx4(d, desc_sw128(a_lo + 6), desc_sw128(b_lo + 6), mx4_idesc<BN>(2), tsa, tsb, 1);
              tsa += 4, tsb += 4 * C::kTilesB;
            }
            mma_commit(freed);
            more = 1;
          }
          if (!ok) break;
          mma_commit(&sempty[q.slot]);
          q.advance();
        }
        any |= more != 0;
        if (!ok) break;
        mma_commit(&tfull[acc.slot]);
        acc.advance();
      }
      if (any) {
        volatile int no_abort = 0;
        mma_commit(drain);
        mbar_wait(drain, 0, &no_abort, kDrainLimitNs);
      }
    }
  } else if (warp < kEpiWarp0) {
    if (warp == 2)  // warp 3 has no role
      schedule_tiles(
          queue, args, [&](uint32_t tiles) { const uint32_t n = args.N / kOutCols; return Mx4Units{tiles * n, n}; },
          lane, abort_word, lim);
  } else if (warp >= kScaleWarp0) {
    regs_dec<kScaleRegs>();
    const uint32_t t_scale = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::kScaleCol0;
    uint32_t q = 0;
    bool ok = true;
    int4 e;
    for (uint32_t i = 0; ok && queue.get(i, e, true, lane, abort_word, lim) && e.x >= 0; ++i) {
      const uint32_t* xs = args.xs + e.y + lane;
      const int rows = args.M - e.y - lane;  // rows from this lane's first on (the tile may reach past M)
      const int n0 = e.w * kOutCols;
      // tiles [Nw/128][KB][512] of this group, 16 bytes a lane; of a unit with
      // 64 gate and 64 up columns half of each tile's words
      const uint8_t* w0 = args.ws + (static_cast<long long>(e.x) * (Nw / 128) + n0 / 128) * KB * 512 + lane * 16 +
                          (kHalfTiles ? (n0 & 64) >> 3 : 0);
      const uint8_t* w1 = w0 + static_cast<long long>(FUSE ? args.N / 128 : 1) * KB * 512;
      for (int k0 = 0; k0 < KB; k0 += kScaleBlocks, ++q) {
        uint32_t v[4 * kScaleBlocks], w[4 * C::kTilesB * kScaleBlocks];
        const bool upper = k0 + 4 < KB;
#pragma unroll
        for (int kb = 0; kb < kScaleBlocks; ++kb) {
          if (kb >= 4 && !upper) break;
          // K blocks past the last one repeat it: stored, but not multiplied
          const long long k = min(k0 + kb, KB - 1);
          const uint32_t* src = xs + k * args.M;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[4 * kb + j] = 32 * j < rows ? __ldg(src + 32 * j) : 0u;
          uint32_t* d = w + 4 * C::kTilesB * kb;
          if (kHalfTiles) {
            const uint2 g = __ldg(reinterpret_cast<const uint2*>(w0 + k * 512));
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(w1 + k * 512));
            d[0] = g.x, d[1] = g.y, d[2] = u.x, d[3] = u.y;
          } else {
#pragma unroll
            for (int n = 0; n < C::kTilesB; ++n) {
              const uint4 g = __ldg(reinterpret_cast<const uint4*>((n ? w1 : w0) + k * 512));
              d[4 * n] = g.x, d[4 * n + 1] = g.y, d[4 * n + 2] = g.z, d[4 * n + 3] = g.w;
            }
          }
        }
        const uint32_t slot = q % kScaleSlots, ph = (q / kScaleSlots) & 1u;
        if (!__all_sync(0xffffffffu, mbar_wait(&sempty[slot], ph ^ 1u, abort_word, lim))) {
          ok = false;
          break;
        }
        tc_fence_after();  // the products that read the slot are done
        const uint32_t t = t_scale + slot * C::kScaleCols;
#pragma unroll
        for (int h = 0; h < kScaleBlocks / 4; ++h) {
          if (h > 0 && !upper) break;
          tmem_st_32x16(t + 16 * h, *reinterpret_cast<uint32_t(*)[16]>(v + 16 * h));
#pragma unroll
          for (int n = 0; n < C::kTilesB; ++n)
            tmem_st_32x16(t + 4 * kScaleBlocks + 16 * (C::kTilesB * h + n),
                          *reinterpret_cast<uint32_t(*)[16]>(w + 16 * (C::kTilesB * h + n)));
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[slot]);
      }
    }
  } else {
    regs_inc<kEpiRegs>();
    const int pw = warp - kEpiWarp0;
    const int half = pw >> 2;
    const int quad = warp & 3;  // TMEM lane quadrant this warp may access
    const int tid = static_cast<int>(threadIdx.x) - 32 * kEpiWarp0;
    const uint32_t t_lane = tbase + (static_cast<uint32_t>(quad * 32) << 16);
    uint8_t* stage = staging + pw * C::kBoxes * 4096;
    const long long N = args.N;
    // rows [S, M) belong to no group: zeros (zero scale bytes too, as
    // quantising zero rows gives)
    const long long S = grouped_rows(args, tid, staging), rest = args.M - S;
    if (rest > 0) {
      const long long first = tid + static_cast<long long>(blockIdx.x) * kEpiThreads;
      const long long step = static_cast<long long>(gridDim.x) * kEpiThreads;
      if (args.out) {
        uint4* p = reinterpret_cast<uint4*>(args.out + S * N);
        for (long long i = first; i < rest * N / 8; i += step) p[i] = make_uint4(0, 0, 0, 0);
      }
      if (MODE == kFusedQuant) {
        uint4* p = reinterpret_cast<uint4*>(args.hq + S * N / 2);
        for (long long i = first; i < rest * N / 32; i += step) p[i] = make_uint4(0, 0, 0, 0);
        for (long long i = first; i < rest * (N / 128); i += step) args.hs[(i / rest) * args.M + S + i % rest] = 0;
      }
    }
    uint32_t t = 0;
    int4 e;
    for (uint32_t i = 0; queue.get(i, e, true, lane, abort_word, lim) && e.x >= 0; ++i) {
      const long long wrow0 = e.y + quad * 32;
      const int nvalid = min(32, e.z - static_cast<int>(wrow0));  // rows of this warp (may be <= 0)
      const int col0 = e.w * kOutCols + half * kWarpCols;
      const uint32_t b = t % kBufs, tph = (t / kBufs) & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[b], tph, abort_word, lim))) break;
      tc_fence_after();
      const uint32_t tb = t_lane + b * BN + half * kWarpCols;
      // the row's part of the accumulator in one go (gate, then up), so that
      // the next unit's products can start
      constexpr int kAcc = FUSE ? 2 * kWarpCols : kWarpCols;
      uint32_t r[kAcc];
#pragma unroll
      for (int cc = 0; cc < kAcc / 32; ++cc)
        tmem_ld_32x32(32 * cc < kWarpCols ? tb + 32 * cc : tb + BN / 2 + 32 * cc - kWarpCols,
                      *reinterpret_cast<uint32_t(*)[32]>(r + 32 * cc));
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[b]);
      ++t;
      if (nvalid <= 0) continue;
      uint32_t v[kWarpCols / 2];  // the row's outputs, bf16 pairs
#pragma unroll
      for (int j = 0; j < kWarpCols / 2; ++j) {
        const float a0 = __uint_as_float(r[2 * j]), a1 = __uint_as_float(r[2 * j + 1]);
        v[j] = FUSE ? pack_bf16x2(silu_f32(a0) * __uint_as_float(r[(kAcc / 2 + 2 * j) % kAcc]),
                                  silu_f32(a1) * __uint_as_float(r[(kAcc / 2 + 2 * j + 1) % kAcc]))
                    : pack_bf16x2(a0, a1);
      }
      if (args.out) {
        if (nvalid == 32 && kWarpCols % 64 == 0) {
          // whole boxes of 32 rows x 64 columns (chunk j of row r at
          // j ^ (r & 7)), one tensor store each
          bulk_wait_read_all();  // this lane's earlier store has read its box
          __syncwarp();
#pragma unroll
          for (int q = 0; q < kWarpCols / 64; ++q)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint4*>(stage + q * 4096 + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                  make_uint4(v[32 * q + 4 * j], v[32 * q + 4 * j + 1], v[32 * q + 4 * j + 2], v[32 * q + 4 * j + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane < kWarpCols / 64) {
            tma_store_2d(&map_out, stage + lane * 4096, col0 + 64 * lane, static_cast<int>(wrow0));
            bulk_commit();
          }
        } else {
          // the rows after this group's are another's: row by row
          using Box = RowBox<2 * kWarpCols <= 128 ? 2 * kWarpCols : 128>;
          constexpr int kParts = 2 * kWarpCols / (Box::kChunks * 16);
          bulk_wait_read_all();
          __syncwarp();
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
#pragma unroll
            for (int j = 0; j < Box::kChunks; ++j) {
              const int c = 4 * (Box::kChunks * q + j);
              Box::put(stage, lane, j, make_uint4(v[c], v[c + 1], v[c + 2], v[c + 3]));
            }
            __syncwarp();
            Box::store(stage, reinterpret_cast<uint8_t*>(args.out + wrow0 * N + col0) + 128 * q, 2 * N, nvalid, lane);
            __syncwarp();
          }
        }
      }
      if (MODE == kFusedQuant) {
        // the row's blocks of 32 lie in one thread: same rule as
        // mx4_quantize_lhs on the bf16 values
        using Box = RowBox<32>;  // codes of 64 columns; of 32, half of it
        uint32_t word = 0;
        if (args.out) bulk_wait_read_all();
        __syncwarp();
#pragma unroll
        for (int q = 0; q < kWarpCols / 32; ++q) {
          uint32_t m2 = 0;
#pragma unroll
          for (int j = 0; j < 16; ++j) m2 = absmax2(m2, v[16 * q + j]);
          const uint32_t byte = mx4_scale_byte(absmax2(m2, m2 >> 16) & 0xffffu);
          const uint32_t inv = mx4_inverse2(byte);
          uint32_t c4[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t part[4] = {v[16 * q + 4 * j], v[16 * q + 4 * j + 1], v[16 * q + 4 * j + 2],
                                      v[16 * q + 4 * j + 3]};
            c4[j] = mx4_codes8(part, inv);
          }
          word |= byte << (8 * q);
          Box::put(stage, lane, q, make_uint4(c4[0], c4[1], c4[2], c4[3]));
        }
        uint8_t* pq = args.hq + (wrow0 * N + col0) / 2;
        if (kWarpCols == 64) {
          __syncwarp();
          Box::store(stage, pq, N / 2, nvalid, lane);
        } else if (lane < nvalid) {
          *reinterpret_cast<uint4*>(pq + lane * (N / 2)) = Box::get(stage, lane, 0);
        }
        __syncwarp();
        if (lane < nvalid) {
          uint8_t* ps = reinterpret_cast<uint8_t*>(args.hs + static_cast<long long>(col0 / 128) * args.M + wrow0 +
                                                   lane) + col0 % 128 / 32;
          if (kWarpCols == 64)
            *reinterpret_cast<uint16_t*>(ps) = static_cast<uint16_t>(word);
          else
            *ps = static_cast<uint8_t>(word);
        }
      }
    }
    bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
  if (threadIdx.x == 0) finish_claims(const_cast<int32_t*>(args.meta), *abort_word != 0);
}

template <int BN, int MODE>
cudaError_t launch(const CUtensorMap& map_a, const CUtensorMap& map_b, const CUtensorMap& map_out,
                   const Mx4Args& args, int grid, cudaStream_t stream) {
  constexpr int smem = Mx4Tile<BN, MODE != kPlain>::kSmemBytes;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(gmm_mx4_kernel<BN, MODE>, smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(gmm_mx4_kernel<BN, MODE>, dim3(grid), dim3(kThreads), smem, stream, map_a, map_b, map_out, args);
}

}  // namespace

cudaError_t launch_gmm_mx4(const CUtensorMap& map_a, const CUtensorMap& map_b, const CUtensorMap& map_out,
                           const Mx4Args& args, int grid, cudaStream_t stream) {
  if (args.bn == 256) {
    if (args.hq) return launch<256, kFusedQuant>(map_a, map_b, map_out, args, grid, stream);
    if (args.fuse) return launch<256, kFused>(map_a, map_b, map_out, args, grid, stream);
    return launch<256, kPlain>(map_a, map_b, map_out, args, grid, stream);
  }
  if (args.hq) return launch<128, kFusedQuant>(map_a, map_b, map_out, args, grid, stream);
  if (args.fuse) return launch<128, kFused>(map_a, map_b, map_out, args, grid, stream);
  return launch<128, kPlain>(map_a, map_b, map_out, args, grid, stream);
}

}  // namespace gmm
