// The gated feed-forward block for training, grouped by expert, in bf16.
//
// Forward: a = x Wgate, b = x Wup (fp32 sums over K), h = bf16(a s(a) b) with
// s the logistic function, and the kept a and b: rounded to bf16, or as e4m3
// codes with one fp32 scale per row and 128 columns (absmax / 448), taken from
// the fp32 sums.
// Backward: dh = dy W2^T (fp32 sums), and with sg = s(a)
//   da = dh b sg (1 + a (1 - sg)),   db = dh a sg,   h = a sg b,
// so dh never goes to memory and h need not be kept: it is recomputed here
// for the second weight's gradient.
//
// Both are one grouped GEMM on the tensor core with the activation in its
// epilogue (384 threads, one persistent CTA per SM):
//   warp 0      TMA: per 64-wide K step the 128 rows of x (or dy) and BN
//               columns of the weight into a ring of shared-memory slots
//   warp 1      TMEM, tcgen05.mma kind::f16 M=128 N=BN K=16, two accumulators,
//               so that one unit's epilogue overlaps the next unit's products
//   warp 2      claims the CTA's units and queues them for the other roles
//   warps 4-11  epilogue: one thread per row and column half
// Rows of a tile past its group's end belong to the next group: they are
// multiplied with the wrong weight and never stored.
#include "common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "unitqueue.cuh"

namespace gmm {

namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kQueueReaders = 2 + kEpiWarps;
constexpr uint64_t kDrainLimitNs = 200000000ull;

template <int BN>
struct SwigluTile {
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr int kABytes = kBM * 64 * 2;
  static constexpr int kBBytes = 64 * BN * 2;
  static constexpr int kBoxBytes = 64 * 64 * 2;  // one 64 x 64 box of the natural-layout weight
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kTmemCols = 2 * BN;
  static constexpr int kBarBytes = 512;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kBarBytes;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static_assert(8 * (2 * kStages + 5 + ClaimQueue::kBarriers) + 16 + 16 * kClaimSlots <= kBarBytes, "barrier area");
};

// s(v) = 1 / (1 + exp(-v)) with the hardware exponential and divide (a few ulp
// of fp32; exp(-v) = inf gives 0)
__device__ __forceinline__ float logistic(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ void unpack8(const uint4& p, float (&v)[8]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// 8 e4m3 codes -> their values times `scale`
__device__ __forceinline__ void unpack8_e4m3(const uint2& p, float scale, float (&v)[8]) {
  const uint32_t w[2] = {p.x, p.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((w[i >> 1] >> (16 * (i & 1))) & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    v[2 * i] = f.x * scale;
    v[2 * i + 1] = f.y * scale;
  }
}

// Zero `bytes` (a multiple of 16) from `p` on, spread over the grid's epilogue threads.
__device__ __forceinline__ void zero_span(void* p, long long bytes, int tid) {
  uint4* q = static_cast<uint4*>(p);
  for (long long i = tid + static_cast<long long>(blockIdx.x) * kEpiThreads; i < bytes / 16;
       i += static_cast<long long>(gridDim.x) * kEpiThreads)
    q[i] = make_uint4(0, 0, 0, 0);
}

// Row `row` of the forward's outputs, 64 columns of h and one 128-column half
// (gate or up) of the kept values, from the accumulators at TMEM address `t`
// (gate in columns [0, 128), up in [128, 256)).
template <bool E4M3>
__device__ __forceinline__ void fwd_row(const SwigluArgs& args, uint32_t t, int half, long long row, bool valid, int n0) {
  const long long N = args.N;
#pragma unroll 1
  for (int cc = 0; cc < 2; ++cc) {
    uint32_t ra[32], rb[32];
    tmem_ld_32x32(t + half * 64 + 32 * cc, ra);
    tmem_ld_32x32(t + 128 + half * 64 + 32 * cc, rb);
    tmem_ld_wait();
    if (valid) {
      const int col = n0 + half * 64 + 32 * cc;
      uint4* ph = reinterpret_cast<uint4*>(args.h + row * N + col);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a[8], b[8], v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = __uint_as_float(ra[8 * j + i]);
          b[i] = __uint_as_float(rb[8 * j + i]);
          v[i] = silu_f32(a[i]) * b[i];
        }
        ph[j] = pack8(v);
        if (!E4M3) {
          reinterpret_cast<uint4*>(args.gu + row * 2 * N + col)[j] = pack8(a);
          reinterpret_cast<uint4*>(args.gu + row * 2 * N + N + col)[j] = pack8(b);
        }
      }
    }
  }
  if (E4M3) {
    // half 0 keeps the gate block, half 1 the up block: absmax, then codes
    // (rounded once, from the fp32 sums)
    const uint32_t tb = t + half * 128;
    float amax = 0.0f;
#pragma unroll 1
    for (int cc = 0; cc < 4; ++cc) {
      uint32_t r[32];
      tmem_ld_32x32(tb + 32 * cc, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(__uint_as_float(r[i])));
    }
    float s, inv;
    e4m3_block_scale(amax, s, inv);
    const long long block = half * (N / 128) + n0 / 128;
    if (valid) args.gus[block * args.M + row] = s;
    uint4* pq = reinterpret_cast<uint4*>(args.guq + row * 2 * N + block * 128);
#pragma unroll 1
    for (int cc = 0; cc < 4; ++cc) {
      uint32_t r[32];
      tmem_ld_32x32(tb + 32 * cc, r);
      tmem_ld_wait();
      if (valid) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t q[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int c = 16 * j + 4 * k;
            q[k] = e4m3x2(__fmul_rn(__uint_as_float(r[c]), inv), __fmul_rn(__uint_as_float(r[c + 1]), inv)) |
                   (e4m3x2(__fmul_rn(__uint_as_float(r[c + 2]), inv), __fmul_rn(__uint_as_float(r[c + 3]), inv))
                    << 16);
          }
          pq[2 * cc + j] = make_uint4(q[0], q[1], q[2], q[3]);
        }
      }
    }
  }
}

// Row `row` of the backward's outputs, BN/2 columns from column `col0`, from
// dh at TMEM address `t`.
template <int BN, bool E4M3>
__device__ __forceinline__ void bwd_row(const SwigluArgs& args, uint32_t t, long long row, bool valid, int col0) {
  const long long N = args.N;
  float sa = 0.0f, sb = 0.0f;
  if (E4M3 && valid) {
    sa = args.gus[static_cast<long long>(col0 / 128) * args.M + row];
    sb = args.gus[static_cast<long long>(N / 128 + col0 / 128) * args.M + row];
  }
#pragma unroll 1
  for (int cc = 0; cc < BN / 64; ++cc) {
    const int col = col0 + 32 * cc;
    uint32_t r[32];
    tmem_ld_32x32(t + 32 * cc, r);
    tmem_ld_wait();
    if (valid) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a[8], b[8], da[8], db[8], hv[8];
        if (E4M3) {
          const uint8_t* p = args.guq + row * 2 * N + col + 8 * j;
          unpack8_e4m3(*reinterpret_cast<const uint2*>(p), sa, a);
          unpack8_e4m3(*reinterpret_cast<const uint2*>(p + N), sb, b);
        } else {
          const uint16_t* p = args.gu + row * 2 * N + col + 8 * j;
          unpack8(*reinterpret_cast<const uint4*>(p), a);
          unpack8(*reinterpret_cast<const uint4*>(p + N), b);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float dh = __uint_as_float(r[8 * j + i]);
          const float sg = logistic(a[i]);
          const float act = a[i] * sg;
          hv[i] = act * b[i];
          db[i] = dh * act;
          da[i] = dh * b[i] * sg * (1.0f + a[i] * (1.0f - sg));
        }
        uint16_t* o = args.dgu + row * 2 * N + col + 8 * j;
        *reinterpret_cast<uint4*>(o) = pack8(da);
        *reinterpret_cast<uint4*>(o + N) = pack8(db);
        if (args.h) *reinterpret_cast<uint4*>(args.h + row * N + col + 8 * j) = pack8(hv);
      }
    }
  }
}

// FWD: W natural [G*K, 2N] (MN-major), units of 128 gate + 128 up columns
// (BN = 256).  Otherwise W2 as rows of its N output columns, K-major, units of
// BN columns.
template <int BN, bool FWD, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1)
    gmm_swiglu_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const SwigluArgs args) {
  static_assert(!FWD || BN == 256, "a forward unit is 128 gate and 128 up columns");
  using C = SwigluTile<BN>;
  constexpr int kStages = C::kStages;
  constexpr int kOutCols = FWD ? 128 : BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + kStages * C::kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
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
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps);
    }
    mbar_init(drain, 1);
    queue.init(kQueueReaders);
    *abort_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_b);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
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
  const int KS = args.K / 64;
  const uint64_t lim = args.wait_limit_ns;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t c = 0;
      bool ok = true;
      int4 e;
      for (uint32_t i = 0; ok && queue.get(i, e, false, 0, abort_word, lim) && e.x >= 0; ++i) {
        const int n0 = e.w * kOutCols;
        for (int ks = 0; ks < KS; ++ks) {
          const uint32_t s = c % kStages, ph = (c / kStages) & 1u;
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_word, lim)) {
            ok = false;
            break;
          }
          uint8_t* a_dst = ring + s * C::kStageBytes;
          uint8_t* b_dst = a_dst + C::kABytes;
          mbar_arrive_expect_tx(&full[s], C::kStageBytes);
          tma_load_2d(a_dst, &map_a, &full[s], ks * 64, e.y);
          if (FWD) {
            const int wrow = e.x * args.K + ks * 64;  // row of the [G*K, 2N] weight view
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tma_load_2d(b_dst + j * C::kBoxBytes, &map_b, &full[s], (j >> 1) * args.N + n0 + 64 * (j & 1), wrow);
          } else {
            tma_load_2d(b_dst, &map_b, &full[s], ks * 64, e.x * args.N + n0);
          }
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
    if (lane == 0) {
      constexpr uint32_t idesc = make_idesc(1u /*bf16*/, false, FWD, kBM, BN);
      uint32_t c = 0, t = 0;
      bool ok = true;
      int4 e;
      for (uint32_t i = 0; ok && queue.get(i, e, false, 0, abort_word, lim) && e.x >= 0; ++i) {
        const uint32_t b = t & 1u, tph = (t >> 1) & 1u;
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
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t bdesc = FWD ? smem_desc_sw128(b_addr + 2048 * j, C::kBoxBytes, 1024)
                                       : smem_desc_sw128(b_addr + 32 * j, 16, 1024);
            mma_bf16(d, smem_desc_sw128(a_addr + 32 * j, 16, 1024), bdesc, idesc, (ks > 0 || j > 0) ? 1u : 0u);
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
    if (lane == 0)
      queue.schedule(args.tiles, const_cast<int32_t*>(args.meta) + kWsClaimed, num_units,
                     static_cast<uint32_t>(per_tile), abort_word, lim);
  } else if (warp >= kEpiWarp0) {
    const int half = (warp - kEpiWarp0) >> 2;
    const int quad = warp & 3;  // TMEM lane quadrant this warp may access
    const int tid = static_cast<int>(threadIdx.x) - 32 * kEpiWarp0;
    const uint32_t t_lane = tbase + (static_cast<uint32_t>(quad * 32) << 16);
    // rows [S, M) belong to no group
    const long long S = args.meta[kWsS], rest = args.M - S, N = args.N;
    if (rest > 0) {
      if (args.h) zero_span(args.h + S * N, rest * N * 2, tid);
      if (!FWD) {
        zero_span(args.dgu + S * 2 * N, rest * N * 4, tid);
      } else if (E4M3) {
        zero_span(args.guq + S * 2 * N, rest * N * 2, tid);
        for (long long i = tid + static_cast<long long>(blockIdx.x) * kEpiThreads; i < rest * (2 * N / 128);
             i += static_cast<long long>(gridDim.x) * kEpiThreads)
          args.gus[(i / rest) * args.M + S + i % rest] = 0.0f;
      } else {
        zero_span(args.gu + S * 2 * N, rest * N * 4, tid);
      }
    }
    uint32_t t = 0;
    int4 e;
    for (uint32_t i = 0; queue.get(i, e, true, lane, abort_word, lim) && e.x >= 0; ++i) {
      const int row = e.y + quad * 32 + lane;
      const bool valid = row < e.z;
      const uint32_t b = t & 1u, tph = (t >> 1) & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[b], tph, abort_word, lim))) break;
      tc_fence_after();
      const uint32_t tb = t_lane + b * BN;
      if (FWD)
        fwd_row<E4M3>(args, tb, half, valid ? row : 0, valid, e.w * 128);
      else
        bwd_row<BN, E4M3>(args, tb + half * (BN / 2), valid ? row : 0, valid, e.w * BN + half * (BN / 2));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[b]);
      ++t;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, C::kTmemCols);
  }
  if (threadIdx.x == 0) finish_claims(const_cast<int32_t*>(args.meta), *abort_word != 0);
}

template <int BN, bool FWD, bool E4M3>
cudaError_t launch(const CUtensorMap& map_a, const CUtensorMap& map_b, const SwigluArgs& args, int grid,
                   cudaStream_t stream) {
  constexpr int smem = SwigluTile<BN>::kSmemBytes;
  cudaError_t e = cudaFuncSetAttribute(gmm_swiglu_kernel<BN, FWD, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(gmm_swiglu_kernel<BN, FWD, E4M3>, dim3(grid), dim3(kThreads), smem, stream, map_a, map_b, args);
}

}  // namespace

cudaError_t launch_gmm_swiglu_fwd(const CUtensorMap& map_x, const CUtensorMap& map_w, const SwigluArgs& args,
                                  int grid, cudaStream_t stream) {
  if (args.guq) return launch<256, true, true>(map_x, map_w, args, grid, stream);
  return launch<256, true, false>(map_x, map_w, args, grid, stream);
}

int swiglu_bwd_bn(int N) { return N % 256 == 0 ? 256 : 128; }

cudaError_t launch_gmm_swiglu_bwd(const CUtensorMap& map_dy, const CUtensorMap& map_w2, const SwigluArgs& args,
                                  int grid, cudaStream_t stream) {
  if (swiglu_bwd_bn(args.N) == 256) {
    if (args.guq) return launch<256, false, true>(map_dy, map_w2, args, grid, stream);
    return launch<256, false, false>(map_dy, map_w2, args, grid, stream);
  }
  if (args.guq) return launch<128, false, true>(map_dy, map_w2, args, grid, stream);
  return launch<128, false, false>(map_dy, map_w2, args, grid, stream);
}

}  // namespace gmm
