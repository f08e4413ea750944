// MXFP4 grouped GEMM: out[m, n] = bf16( sum over blocks of 32 along K of
//   2^(sx - 127) 2^(sw - 127) sum_k cx[m, k] cw[g, n, k] ),  m in group g,
// on the block-scaled tensor core (kind::mxf4: packed E2M1 operands, E8M0
// scales applied in the product, fp32 sums).  With a gate | up weight the
// output is silu(gate) * up, as bf16 and / or as MXFP4 for the next product.
//
// 384 threads, one persistent CTA per SM, units of 128 rows x BN weight columns:
//   warp 0      TMA: per K step of 256 (128 packed bytes a row) the codes of
//               128 rows and of BN columns into a ring slot
//   warp 1      copies the slot's scales into tensor memory (tcgen05.cp, one
//               per 128 rows x 128 of K), then four tcgen05.mma of K = 64
//   warp 2      fetches the slot's scales (cp.async).  A tile of 128 rows x 128
//               of K is 512 bytes, row r's four bytes at (r % 32) * 16 +
//               (r / 32) * 4: weights are stored so, activations are not (a
//               group starts at any row), so lane l gathers rows l, l + 32, ...
//   warp 3      claims the CTA's units and queues them for the other roles
//   warps 4-11  epilogue
// BN = 256 fills half of the tensor memory with one accumulator and needs the
// rest for the scales, so the epilogue's loads stop the products of the next
// unit (its operands are fetched meanwhile); BN = 128 has two accumulators.
#include "common.cuh"
#include "kernels.cuh"
#include "mx4.cuh"
#include "ptx.cuh"
#include "unitqueue.cuh"

namespace gmm {

namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kQueueReaders = 3 + kEpiWarps;
constexpr uint64_t kDrainLimitNs = 200000000ull;

enum Mx4Mode { kPlain = 0, kFused = 1, kFusedQuant = 2 };

template <int BN>
struct Mx4Tile {
  static constexpr int kStages = BN == 256 ? 3 : 4;
  static constexpr int kBufs = BN == 256 ? 1 : 2;
  static constexpr int kABytes = kBM * 128;
  static constexpr int kBBytes = BN * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kTilesB = BN / 128;                      // 128-column scale tiles
  static constexpr int kScaleBytes = 2 * 512 * (1 + kTilesB);   // two 128-wide K blocks
  static constexpr int kScaleCol0 = 256;                        // first tensor-memory column of the scales
  static constexpr int kScaleCols = 32;                         // columns per ring slot
  static constexpr int kBoxes = BN / 128;                       // 32 x 64 staging boxes per warp
  static constexpr int kStagingBytes = kEpiWarps * kBoxes * 4096;
  static constexpr int kBarBytes = 512;
  static constexpr int kSmemBytes = 1024 + kStages * (kStageBytes + kScaleBytes) + kStagingBytes + kBarBytes;
  static_assert(kBufs * BN <= kScaleCol0 && kScaleCol0 + kStages * kScaleCols <= 512, "tensor memory");
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static_assert(8 * (2 * kStages + 2 * kBufs + 1 + ClaimQueue::kBarriers) + 16 + 16 * kClaimSlots <= kBarBytes,
                "barrier area");
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
  using C = Mx4Tile<BN>;
  constexpr bool FUSE = MODE != kPlain;
  constexpr int kStages = C::kStages, kBufs = C::kBufs;
  constexpr int kOutCols = FUSE ? BN / 2 : BN;
  constexpr int kWarpCols = kOutCols / 2;  // output columns per epilogue warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* staging = ring + kStages * C::kStageBytes;
  uint8_t* scales = staging + C::kStagingBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + kStages * C::kScaleBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
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
      mbar_init(&full[s], 2);  // the codes' copies, and the scales
      mbar_init(&empty[s], 1);
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

  const int per_tile = args.N / kOutCols;
  const uint32_t num_units = static_cast<uint32_t>(args.meta[kWsNumTiles]) * static_cast<uint32_t>(per_tile);
  const int KB = args.K / 128, KS = (KB + 1) / 2;
  const int Nw = FUSE ? 2 * args.N : args.N;
  const uint64_t lim = args.wait_limit_ns;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t c = 0;
      bool ok = true;
      int4 e;
      for (uint32_t i = 0; ok && queue.get(i, e, false, 0, abort_word, lim) && e.x >= 0; ++i) {
        const int brow = e.x * Nw + e.w * kOutCols;
        for (int ks = 0; ks < KS; ++ks) {
          const uint32_t s = c % kStages, ph = (c / kStages) & 1u;
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_word, lim)) {
            ok = false;
            break;
          }
          uint8_t* a_dst = ring + s * C::kStageBytes;
          uint8_t* b_dst = a_dst + C::kABytes;
          // past K (an odd number of 128-wide blocks) the copies bring zeros
          mbar_arrive_expect_tx(&full[s], C::kStageBytes);
          tma_load_2d(a_dst, &map_a, &full[s], ks * 128, e.y);
          tma_load_2d(b_dst, &map_b, &full[s], ks * 128, brow);
          if (FUSE) tma_load_2d(b_dst + C::kBBytes / 2, &map_b, &full[s], ks * 128, brow + args.N);
          ++c;
        }
      }
      // wait for the last copy issued into every slot (its barrier phase also
      // needs the scales; when that role has given up, the copies have long
      // landed by the time this wait runs out)
      volatile int no_abort = 0;
      for (uint32_t s = 0; s < kStages; ++s) {
        if (c > s) {
          const uint32_t last = s + kStages * ((c - 1 - s) / kStages);
          mbar_wait(&full[s], (last / kStages) & 1u, &no_abort, kDrainLimitNs);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t c = 0, t = 0;
      bool ok = true;
      int4 e;
      for (uint32_t i = 0; ok && queue.get(i, e, false, 0, abort_word, lim) && e.x >= 0; ++i) {
        const uint32_t b = t % kBufs, tph = (t / kBufs) & 1u;
        if (!mbar_wait(&tempty[b], tph ^ 1u, abort_word, lim)) break;
        const uint32_t d = tbase + b * BN;
        for (int ks = 0; ks < KS; ++ks) {
          const uint32_t s = c % kStages, ph = (c / kStages) & 1u;
          if (!mbar_wait(&full[s], ph, abort_word, lim)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(ring + s * C::kStageBytes);
          const uint32_t b_addr = a_addr + C::kABytes;
          const uint32_t sc = smem_u32(scales + s * C::kScaleBytes);
          // slot's scale columns: A's two K blocks (4 columns each), then B's
          const uint32_t tsa = tbase + C::kScaleCol0 + s * C::kScaleCols, tsb = tsa + 8;
          const int blocks = min(2, KB - 2 * ks);
#pragma unroll
          for (int kb = 0; kb < 2; ++kb) {
            if (kb < blocks) {
              tmem_cp_scales(tsa + 4 * kb, smem_desc_rows16(sc + 512 * kb));
#pragma unroll
              for (int q = 0; q < C::kTilesB; ++q)
                tmem_cp_scales(tsb + 4 * (C::kTilesB * kb + q), smem_desc_rows16(sc + 1024 + 512 * (C::kTilesB * kb + q)));
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j < 2 * blocks)
              mma_mx4(d, smem_desc_sw128(a_addr + 32 * j, 16, 1024), smem_desc_sw128(b_addr + 32 * j, 16, 1024),
                      mx4_idesc<BN>(2 * (j & 1)), tsa + 4 * (j >> 1), tsb + 4 * C::kTilesB * (j >> 1),
                      (ks > 0 || j > 0) ? 1u : 0u);
          }
          mma_commit(&empty[s]);
          ++c;
        }
        if (!ok) break;
        mma_commit(&tfull[b]);
        ++t;
      }
      if (c > 0) {
        volatile int no_abort = 0;
        mma_commit(drain);
        mbar_wait(drain, 0, &no_abort, kDrainLimitNs);
      }
    }
  } else if (warp == 2) {
    // The slot's arrival lags its copies by kLag steps, so that kLag steps'
    // scales are in flight.  kLag < kStages: a slot is waited for only after
    // the step that frees it has been handed over.
    constexpr uint32_t kLag = 2;
    uint32_t c = 0, handed = 0;
    bool ok = true;
    int4 e;
    for (uint32_t i = 0; ok && queue.get(i, e, true, lane, abort_word, lim) && e.x >= 0; ++i) {
      const uint32_t* xs = args.xs + e.y;
      const int n0 = e.w * kOutCols;
      for (int ks = 0; ks < KS; ++ks) {
        const uint32_t s = c % kStages, ph = (c / kStages) & 1u;
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1u, abort_word, lim))) {
          ok = false;
          break;
        }
        uint8_t* dst = scales + s * C::kScaleBytes + lane * 16;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          const int k = 2 * ks + kb;
          if (k < KB) {
            const uint32_t* src = xs + static_cast<long long>(k) * args.M;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (e.y + 32 * j + lane < args.M) cp_async_4(dst + 512 * kb + 4 * j, src + 32 * j + lane);
            // weight column tiles: [Nw/128][KB][512] bytes of this group
            const uint8_t* wg = args.ws + (static_cast<long long>(e.x) * (Nw / 128) * KB + k) * 512 + lane * 16;
            uint8_t* db = dst + 1024 + 512 * C::kTilesB * kb;
            if (FUSE && BN == 128) {
              // 64 gate and 64 up columns: half a tile of each
              const int off = (n0 & 64) >> 3;  // 8 bytes: the upper 64 columns' words
              cp_async_8(db, wg + static_cast<long long>(n0 / 128) * KB * 512 + off);
              cp_async_8(db + 8, wg + static_cast<long long>((args.N + n0) / 128) * KB * 512 + off);
            } else {
#pragma unroll
              for (int q = 0; q < C::kTilesB; ++q)
                cp_async_16(db + 512 * q,
                            wg + static_cast<long long>((n0 + (q ? (FUSE ? args.N : 128) : 0)) / 128) * KB * 512);
            }
          }
        }
        cp_async_commit();
        ++c;
        if (c - handed > kLag) {
          cp_async_wait_group<kLag>();
          fence_proxy_async_smem();  // the tensor core's copies read the scales
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[handed % kStages]);
          ++handed;
        }
      }
    }
    // The last kLag steps.  (Until here they may wait for the next unit's
    // entry: the scheduler writes it without waiting for their products.)
    cp_async_wait_group<0>();
    fence_proxy_async_smem();
    __syncwarp();
    for (; handed < c; ++handed)
      if (lane == 0) mbar_arrive(&full[handed % kStages]);
  } else if (warp == 3) {
    if (lane == 0)
      queue.schedule(args.tiles, const_cast<int32_t*>(args.meta) + kWsClaimed, num_units,
                     static_cast<uint32_t>(per_tile), abort_word, lim);
  } else {
    const int pw = warp - kEpiWarp0;
    const int half = pw >> 2;
    const int quad = warp & 3;  // TMEM lane quadrant this warp may access
    const int tid = static_cast<int>(threadIdx.x) - 32 * kEpiWarp0;
    const uint32_t t_lane = tbase + (static_cast<uint32_t>(quad * 32) << 16);
    uint8_t* stage = staging + pw * C::kBoxes * 4096;
    const long long N = args.N;
    // rows [S, M) belong to no group: zeros (zero scale bytes too, as
    // quantising zero rows gives)
    const long long S = args.meta[kWsS], rest = args.M - S;
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
      const int wrow0 = e.y + quad * 32;
      const int nvalid = min(32, e.z - wrow0);  // rows of this warp (may be <= 0)
      const int col0 = e.w * kOutCols + half * kWarpCols;
      const uint32_t b = t % kBufs, tph = (t / kBufs) & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[b], tph, abort_word, lim))) break;
      tc_fence_after();
      const uint32_t tb = t_lane + b * BN + half * kWarpCols;
      uint32_t v[kWarpCols / 2];  // this row's kWarpCols outputs, bf16 pairs
#pragma unroll
      for (int cc = 0; cc < kWarpCols / 32; ++cc) {
        uint32_t r[32];
        tmem_ld_32x32(tb + 32 * cc, r);
        if (FUSE) {
          uint32_t u[32];
          tmem_ld_32x32(tb + BN / 2 + 32 * cc, u);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[16 * cc + j] = pack_bf16x2(silu_f32(__uint_as_float(r[2 * j])) * __uint_as_float(u[2 * j]),
                                         silu_f32(__uint_as_float(r[2 * j + 1])) * __uint_as_float(u[2 * j + 1]));
        } else {
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[16 * cc + j] = pack_bf16x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[b]);
      ++t;
      if (nvalid <= 0) continue;
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
            tma_store_2d(&map_out, stage + lane * 4096, col0 + 64 * lane, wrow0);
            bulk_commit();
          }
        } else if (lane < nvalid) {
          // the rows after this group's are another's: plain stores
          uint4* p = reinterpret_cast<uint4*>(args.out + (wrow0 + lane) * N + col0);
#pragma unroll
          for (int j = 0; j < kWarpCols / 8; ++j)
            p[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      }
      if (MODE == kFusedQuant && lane < nvalid) {
        // the row's blocks of 32 lie in one thread: same rule as
        // mx4_quantize_lhs on the bf16 values
        const long long row = wrow0 + lane;
        uint8_t* pq = args.hq + (row * N + col0) / 2;
        uint8_t* ps = reinterpret_cast<uint8_t*>(args.hs + static_cast<long long>(col0 / 128) * args.M + row) +
                      col0 % 128 / 32;
#pragma unroll
        for (int q = 0; q < kWarpCols / 32; ++q) {
          uint32_t m2 = 0;
#pragma unroll
          for (int j = 0; j < 16; ++j) m2 = absmax2(m2, v[16 * q + j]);
          const uint32_t byte = mx4_scale_byte(max(m2 & 0xffffu, m2 >> 16));
          const float inv = mx4_inverse(byte);
          uint32_t c4[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t part[4] = {v[16 * q + 4 * j], v[16 * q + 4 * j + 1], v[16 * q + 4 * j + 2],
                                      v[16 * q + 4 * j + 3]};
            c4[j] = mx4_codes8(part, inv);
          }
          *reinterpret_cast<uint4*>(pq + 16 * q) = make_uint4(c4[0], c4[1], c4[2], c4[3]);
          ps[q] = static_cast<uint8_t>(byte);
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
  constexpr int smem = Mx4Tile<BN>::kSmemBytes;
  cudaError_t e =
      cudaFuncSetAttribute(gmm_mx4_kernel<BN, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
