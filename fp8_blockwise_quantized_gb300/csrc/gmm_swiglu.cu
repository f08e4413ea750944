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
//   warp 0      TMA: per 64-wide K step the 128 rows of x (or dy) and the unit's
//               columns of the weight into a ring of shared-memory slots
//   warp 1      TMEM, tcgen05.mma kind::f16 M=128 K=16, two accumulators, so that
//               one unit's epilogue overlaps the next unit's products
//   warp 2      claims the CTA's units and queues them for the other roles
//   warps 4-11  epilogue: one thread per row and column half.  The forward's
//               adds up sums over 512 of K in registers; where gate | up are
//               kept in e4m3, the two threads of a row exchange their halves'
//               largest values
// Rows of a tile past its group's end belong to the next group: they are
// multiplied with the wrong weight and never stored.
//
// Both are bound by memory at the production shape (256 experts, 65536 rows, K
// 2048, N 512, Zipf routing; cold L2).  Forward, e4m3 kept: 291 us, 5.0 TB/s of
// algorithmic bytes, 0.94 PFLOP/s (bf16 kept 295), bound by the operands that reach the SMs (4.0
// GB through L2, 1.3 GB of them from HBM): its loads alone take 237, its products
// alone 162.  Backward, bf16 kept: 206 us, 5.5 TB/s, bound by HBM (without its
// epilogue 161).  256 weight columns a unit, because every unit reads its 128
// rows again.
#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rowbox.cuh"
#include "unitqueue.cuh"

namespace gmm {

namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kQueueReaders = 2 + kEpiWarps;
constexpr uint64_t kDrainLimitNs = 200000000ull;
// Register split: 168 per thread at launch; the epilogue warpgroups hold a
// 32-column piece of four tensors and the next one's inputs.
constexpr uint32_t kControlRegs = 72, kEpiRegs = 216;
static_assert(128 * kControlRegs + 256 * kEpiRegs <= kThreads * 168, "register split exceeds the launch budget");

constexpr int kStages = 4;
constexpr int kABytes = kBM * 64 * 2;
constexpr int kHalfB = 128 * 64 * 2;        // 128 weight columns of a K step
constexpr int kBoxBytes = 64 * 64 * 2;      // one 64 x 64 box of the natural-layout weight
constexpr int kStageBytes = kABytes + 2 * kHalfB;
constexpr int kStagingBytes = kEpiWarps * 4096;
constexpr int kBarBytes = 512;
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kStagingBytes + kBarBytes;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
static_assert(8 * (2 * kStages + 5 + ClaimQueue::kBarriers + kEpiWarps / 2) + 16 + 16 * kClaimSlots <= kBarBytes,
              "barrier area");
// K steps of the forward whose products the tensor core adds up by itself (512
// of K); the epilogue adds these sums in fp32 registers.  The tensor core's adder
// truncates, and a sum of 128 of its steps (K 2048) came out 2.3e-6 low, one of
// 256 (K 4096) twice that, where fp32 products with rounding are 0.6e-6 and
// 0.9e-6 off: the scales of the 8-bit checkpoint show it.  With 512 of K a sum
// they are 0.55e-6 off for any K.  It costs 1 % (65536 rows, K 2048: 294 us, 291
// with one sum for all of K).  The backward's results are all bf16.
constexpr int kSumSteps = 8;

// The work units.  A wide unit is 128 rows x 256 weight columns (forward: 128
// gate and 128 up columns; backward: 256 columns of dh), a narrow one half of
// that.  Units are wide, but where the last round of wide ones would leave half
// of the CTAs or more without any, its units are cut in two: a narrow unit
// takes a little over half a wide one's time (32 experts, 8192 rows, K 2048, N
// 512, cold L2: backward 49.8 us, with wide units only 54.0; forward 58.0 and
// 60.1).
// Widths are fixed to wide for the forward's e4m3 output (a scale covers a
// unit's 128 columns) and to narrow where N is not a multiple of 256 in the
// backward.
struct Units {
  uint32_t wide;      // units [0, wide) are wide
  uint32_t num;       // units in all
  uint32_t per_tile;  // wide units (narrow ones when there are no wide ones) per row tile
  bool all_narrow;
  __device__ Units(uint32_t tiles, int N, bool fwd, bool can_wide, bool can_narrow) {
    const uint32_t wide_cols = fwd ? 128 : 256;
    all_narrow = !can_wide;
    per_tile = all_narrow ? N / (wide_cols / 2) : N / wide_cols;
    num = tiles * per_tile;
    wide = all_narrow ? 0 : num;
    if (!all_narrow && can_narrow) {
      const uint32_t rest = num % gridDim.x;
      if (2 * rest <= gridDim.x) {
        wide = num - rest;
        num += rest;
      }
    }
  }
  // row tile, and the first half-unit column with the width (1 narrow, 2 wide)
  // in the low bits
  __device__ uint2 at(uint32_t u) const {
    if (all_narrow) return make_uint2(u / per_tile, (u % per_tile) << 2 | 1);
    if (u < wide) return make_uint2(u / per_tile, (2 * (u % per_tile)) << 2 | 2);
    const uint32_t v = u - wide, w = wide + v / 2;
    return make_uint2(w / per_tile, (2 * (w % per_tile) + (v & 1)) << 2 | 1);
  }
};

// s(v) = 1 / (1 + exp(-v)) with the hardware exponential and divide (a few ulp
// of fp32; exp(-v) = inf gives 0)
__device__ __forceinline__ float logistic(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

__device__ __forceinline__ void unpack8(const uint4& p, float* v) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// 8 e4m3 codes -> their values times `scale`
__device__ __forceinline__ void unpack8_e4m3(const uint2& p, float scale, float* v) {
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

// The epilogues of one warp: `rows` (1..32) rows from `row0` on, this lane's row
// in tensor memory at `t`; `stage` is the warp's 4 KB of shared memory.
using Box64 = RowBox<64>;  // 32 rows x 32 bf16, or 64 codes
using Box32 = RowBox<32>;  // 32 rows x 32 codes

__device__ __forceinline__ void put32(uint8_t* box, int lane, const float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    Box64::put(box, lane, j,
               make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                          pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7])));
}

// Forward: the sums of one thread's row, half of the unit's gate columns (from
// column half * cols / 2 on) and the same half of its up columns, 32 or 64 each.
struct FwdSums {
  float a[64], b[64];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 64; ++i) a[i] = b[i] = 0.0f;
  }
  // adds the chunk's accumulators: gate in columns [0, cols), up in [cols, 2 cols)
  __device__ __forceinline__ void add(uint32_t t, int half, int cols) {
    const uint32_t ta = t + half * (cols / 2), tb = ta + cols;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (p == 1 && cols < 128) break;
      uint32_t r[32];
      tmem_ld_32x32(ta + 32 * p, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) a[32 * p + i] += __uint_as_float(r[i]);
      tmem_ld_32x32(tb + 32 * p, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) b[32 * p + i] += __uint_as_float(r[i]);
    }
  }
};

__device__ __forceinline__ float absmax64(const float (&v)[64]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 64; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// This lane's 64 sums as e4m3 codes (rounded once, from the fp32 sums) to `g`.
__device__ __forceinline__ void store_codes64(uint8_t* box, uint8_t* g, long long ld, int rows, int lane,
                                              const float (&v)[64], float inv) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = 16 * j + 4 * k;
      q[k] = e4m3x2(__fmul_rn(v[c], inv), __fmul_rn(v[c + 1], inv)) |
             (e4m3x2(__fmul_rn(v[c + 2], inv), __fmul_rn(v[c + 3], inv)) << 16);
    }
    Box64::put(box, lane, j, make_uint4(q[0], q[1], q[2], q[3]));
  }
  __syncwarp();
  Box64::store(box, g, ld, rows, lane);
  __syncwarp();
}

// The two warps that hold the halves of 32 rows exchange the halves' largest
// values: mine and the other's (two slots each, by the unit's parity) and a
// barrier at which both arrive.  Neither can arrive for the next unit before the
// other has, which it does after reading this unit's slot: so the barrier is at
// most one phase ahead of a waiting warp, and a slot written again two units
// later has been read.
struct HalfMax {
  float2 *mine, *other;
  uint64_t* both;
  __device__ __forceinline__ void say(uint32_t unit, int lane, float a, float b) const {
    mine[32 * (unit & 1u) + lane] = make_float2(a, b);
    __syncwarp();
    if (lane == 0) mbar_arrive(both);
  }
  __device__ __forceinline__ bool hear(uint32_t unit, int lane, float& a, float& b, volatile int* abort_word,
                                       uint64_t lim) const {
    if (!__all_sync(0xffffffffu, mbar_wait(both, unit & 1u, abort_word, lim))) return false;
    const float2 v = other[32 * (unit & 1u) + lane];
    __syncwarp();
    a = fmaxf(a, v.x);
    b = fmaxf(b, v.y);
    return true;
  }
};

// Forward, gate | up kept in bf16: half of the unit's `cols` (64 or 128) columns.
__device__ __forceinline__ void fwd_rows_bf16(const SwigluArgs& args, uint8_t* stage, const FwdSums& s, int half,
                                              int lane, long long row0, int rows, int n0, int cols) {
  const long long N = args.N;
  uint8_t* box0 = stage;
  uint8_t* box1 = stage + Box64::kBytes;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    if (p == 1 && cols < 128) break;
    const int col = n0 + half * (cols / 2) + 32 * p;
    put32(box0, lane, s.a + 32 * p);
    put32(box1, lane, s.b + 32 * p);
    __syncwarp();
    uint8_t* g = reinterpret_cast<uint8_t*>(args.gu + row0 * 2 * N + col);
    Box64::store(box0, g, 4 * N, rows, lane);
    Box64::store(box1, g + 2 * N, 4 * N, rows, lane);
    __syncwarp();
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = silu_f32(s.a[32 * p + i]) * s.b[32 * p + i];
    put32(box0, lane, v);
    __syncwarp();
    Box64::store(box0, reinterpret_cast<uint8_t*>(args.h + row0 * N + col), 2 * N, rows, lane);
    __syncwarp();
  }
}

// Forward, gate | up kept in e4m3: 64 of the block's 128 columns, unit number
// `unit` of this warp that has rows.  False: a wait ran out.
__device__ __forceinline__ bool fwd_rows_e4m3(const SwigluArgs& args, uint8_t* stage, const HalfMax& halves,
                                              const FwdSums& s, int half, int lane, long long row0, int rows, int n0,
                                              uint32_t unit, volatile int* abort_word, uint64_t lim) {
  const long long N = args.N;
  float amax = absmax64(s.a), bmax = absmax64(s.b);
  halves.say(unit, lane, amax, bmax);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = silu_f32(s.a[32 * p + i]) * s.b[32 * p + i];
    put32(stage, lane, v);
    __syncwarp();
    Box64::store(stage, reinterpret_cast<uint8_t*>(args.h + row0 * N + n0 + 64 * half + 32 * p), 2 * N, rows, lane);
    __syncwarp();
  }
  if (!halves.hear(unit, lane, amax, bmax, abort_word, lim)) return false;
  float sa, ia, sb, ib;
  e4m3_block_scale(amax, sa, ia);
  e4m3_block_scale(bmax, sb, ib);
  if (lane < rows) args.gus[(half * (N / 128) + n0 / 128) * args.M + row0 + lane] = half ? sb : sa;
  uint8_t* g = args.guq + row0 * 2 * N + n0 + 64 * half;
  store_codes64(stage, g, 2 * N, rows, lane, s.a, ia);
  store_codes64(stage, g + N, 2 * N, rows, lane, s.b, ib);
  return true;
}

// Backward: 32 columns at a time of the kept gate and up.
template <bool E4M3>
struct Kept32 {
  using Box = std::conditional_t<E4M3, Box32, Box64>;
  uint4 a[Box::kSweeps], b[Box::kSweeps];
  __device__ __forceinline__ void fetch(const SwigluArgs& args, long long row0, int rows, int col, int lane) {
    const long long N = args.N;
    constexpr int kElem = E4M3 ? 1 : 2;
    const uint8_t* g = (E4M3 ? args.guq : reinterpret_cast<const uint8_t*>(args.gu)) + (row0 * 2 * N + col) * kElem;
    Box::fetch(a, g, 2 * N * kElem, rows, lane);
    Box::fetch(b, g + N * kElem, 2 * N * kElem, rows, lane);
  }
};

// Backward: `cols` columns from `col0` on, dh at tensor memory address `t`;
// `next` holds the first 32 columns of the kept values.
template <bool E4M3>
__device__ __forceinline__ void bwd_rows(const SwigluArgs& args, uint8_t* stage, uint32_t t, int lane, long long row0,
                                         int rows, int col0, int cols, Kept32<E4M3>& next, float sa,
                                         float sb) {
  using Box = typename Kept32<E4M3>::Box;
  const long long N = args.N, ldh = 2 * N, ldg = 4 * N;
  uint8_t* box0 = stage;
  uint8_t* box1 = stage + Box64::kBytes;
#pragma unroll 1
  for (int cc = 0; cc < cols / 32; ++cc) {
    const int col = col0 + 32 * cc;
    Box::put_sweeps(box0, next.a, lane);
    Box::put_sweeps(box1, next.b, lane);
    __syncwarp();
    float a[32], b[32];
    if (E4M3) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 ca = Box32::get(box0, lane, j), cb = Box32::get(box1, lane, j);
        unpack8_e4m3(make_uint2(ca.x, ca.y), sa, a + 16 * j);
        unpack8_e4m3(make_uint2(ca.z, ca.w), sa, a + 16 * j + 8);
        unpack8_e4m3(make_uint2(cb.x, cb.y), sb, b + 16 * j);
        unpack8_e4m3(make_uint2(cb.z, cb.w), sb, b + 16 * j + 8);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        unpack8(Box64::get(box0, lane, j), a + 8 * j);
        unpack8(Box64::get(box1, lane, j), b + 8 * j);
      }
    }
    __syncwarp();
    if (cc + 1 < cols / 32) next.fetch(args, row0, rows, col + 32, lane);
    uint32_t r[32];
    tmem_ld_32x32(t + 32 * cc, r);
    tmem_ld_wait();
    float da[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float dh = __uint_as_float(r[i]);
      const float sg = logistic(a[i]);
      const float act = a[i] * sg;
      da[i] = dh * b[i] * sg * (1.0f + a[i] * (1.0f - sg));
      a[i] = dh * act;    // up's gradient
      b[i] = act * b[i];  // h
    }
    put32(box0, lane, da);
    put32(box1, lane, a);
    __syncwarp();
    uint8_t* g = reinterpret_cast<uint8_t*>(args.dgu + row0 * 2 * N + col);
    Box64::store(box0, g, ldg, rows, lane);
    Box64::store(box1, g + 2 * N, ldg, rows, lane);
    __syncwarp();
    if (args.h) {
      put32(box0, lane, b);
      __syncwarp();
      Box64::store(box0, reinterpret_cast<uint8_t*>(args.h + row0 * N + col), ldh, rows, lane);
      __syncwarp();
    }
  }
}

// FWD: W natural [G*K, 2N] (MN-major).  Otherwise W2 as rows of its N output
// columns, K-major.
template <bool FWD, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1)
    gmm_swiglu_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const SwigluArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* staging = ring + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kStagingBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* ufull = drain + 1;
  uint64_t* uempty = ufull + kClaimSlots;
  uint64_t* halves = uempty + kClaimSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(halves + kEpiWarps / 2);
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
    for (int q = 0; q < kEpiWarps / 2; ++q) mbar_init(&halves[q], 2);
    queue.init(kQueueReaders);
    *abort_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_b);
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

  const int KS = args.K / 64;
  const int chunk = FWD ? kSumSteps : KS;
  const uint64_t lim = args.wait_limit_ns;

  if (warp < kEpiWarp0) regs_dec<kControlRegs>();
  if (warp == 0) {
    if (lane == 0) {
      RingPos<kStages> r;
      uint32_t c = 0;
      bool ok = true;
      int4 e;
      for (uint32_t i = 0; ok && queue.get(i, e, false, 0, abort_word, lim) && e.x >= 0; ++i) {
        const int width = e.w & 3, n0 = (e.w >> 2) * (FWD ? 64 : 128);
        for (int ks = 0; ks < KS; ++ks) {
          if (!mbar_wait(&empty[r.slot], r.phase ^ 1u, abort_word, lim)) {
            ok = false;
            break;
          }
          uint8_t* dst = ring + r.slot * kStageBytes;
          uint64_t* bar = &full[r.slot];
          mbar_arrive_expect_tx(bar, kABytes + width * kHalfB);
          tma_load_2d(dst, &map_a, bar, ks * 64, e.y);
          dst += kABytes;
          if (FWD) {
            // gate boxes, then up boxes, of 64 columns
            const int wrow = e.x * args.K + ks * 64;  // row of the [G*K, 2N] weight view
            tma_load_2d(dst, &map_b, bar, n0, wrow);
            if (width == 2) tma_load_2d(dst + kBoxBytes, &map_b, bar, n0 + 64, wrow);
            dst += width * kBoxBytes;
            tma_load_2d(dst, &map_b, bar, args.N + n0, wrow);
            if (width == 2) tma_load_2d(dst + kBoxBytes, &map_b, bar, args.N + n0 + 64, wrow);
          } else {
            tma_load_2d(dst, &map_b, bar, ks * 64, e.x * args.N + n0);
            if (width == 2) tma_load_2d(dst + kHalfB, &map_b, bar, ks * 64, e.x * args.N + n0 + 128);
          }
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
      constexpr uint32_t idesc1 = make_idesc(1u /*bf16*/, false, FWD, kBM, 128);
      constexpr uint32_t idesc2 = make_idesc(1u /*bf16*/, false, FWD, kBM, 256);
      const uint32_t a_lo0 = desc_lo_sw128(smem_u32(ring), 16);
      const uint32_t b_lo0 = desc_lo_sw128(smem_u32(ring) + kABytes, FWD ? kBoxBytes : 16);
      constexpr uint32_t kBStep = (FWD ? 2048 : 32) >> 4;
      RingPos<kStages> r;
      RingPos<2> acc;
      bool ok = true, any = false, next_ready = false;
      int4 e;
      for (uint32_t i = 0; ok && queue.get(i, e, false, 0, abort_word, lim) && e.x >= 0; ++i) {
        const uint32_t idesc = (e.w & 3) == 2 ? idesc2 : idesc1;
        for (int k0 = 0; ok && k0 < KS; k0 += chunk) {
          if (!mbar_wait(&tempty[acc.slot], acc.phase ^ 1u, abort_word, lim)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tbase + acc.slot * 256;
          const int k1 = min(KS, k0 + chunk);
          for (int ks = k0; ks < k1; ++ks) {
            if (!next_ready && !mbar_wait(&full[r.slot], r.phase, abort_word, lim)) {
              ok = false;
              break;
            }
            const uint32_t a_lo = a_lo0 + r.slot * (kStageBytes >> 4);
            const uint32_t b_lo = b_lo0 + r.slot * (kStageBytes >> 4);
            uint64_t* freed = &empty[r.slot];
            r.advance();
            next_ready = mbar_test(&full[r.slot], r.phase);  // answered while the products are issued
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
              mma_bf16(d, desc_sw128(a_lo + 2 * j), desc_sw128(b_lo + kBStep * j), idesc, (ks > k0 || j > 0) ? 1u : 0u);
            mma_commit(freed);
            any = true;
          }
          if (!ok) break;
          mma_commit(&tfull[acc.slot]);
          acc.advance();
        }
      }
      if (any) {
        volatile int no_abort = 0;
        mma_commit(drain);
        mbar_wait(drain, 0, &no_abort, kDrainLimitNs);
      }
    }
  } else if (warp == 2) {
    schedule_tiles(
        queue, args,
        [&](uint32_t tiles) { return Units(tiles, args.N, FWD, FWD || args.N % 256 == 0, !FWD || !E4M3); }, lane,
        abort_word, lim);
  } else if (warp >= kEpiWarp0) {
    regs_inc<kEpiRegs>();
    const int half = (warp - kEpiWarp0) >> 2;
    const int quad = warp & 3;  // TMEM lane quadrant this warp may access
    const int tid = static_cast<int>(threadIdx.x) - 32 * kEpiWarp0;
    const uint32_t t_lane = tbase + (static_cast<uint32_t>(quad * 32) << 16);
    // rows [S, M) belong to no group
    const long long S = grouped_rows(args, tid, staging), rest = args.M - S, N = args.N;
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
    uint8_t* stage = staging + (warp - kEpiWarp0) * 4096;
    RingPos<2> acc;
    int4 e;
    bool ok = true;
    if (FWD) {
      const int pw = warp - kEpiWarp0, po = pw ^ 4;  // po holds the other half of these rows (pw % 4 = quad)
      float2* maxima = reinterpret_cast<float2*>(staging + Box64::kBytes);  // the e4m3 form leaves the second box free
      const HalfMax halves_of_rows{maxima + pw * 512, maxima + po * 512, &halves[quad]};
      uint32_t units = 0;  // with rows, so far
      FwdSums sums;
      for (uint32_t i = 0; ok && queue.get(i, e, true, lane, abort_word, lim) && e.x >= 0; ++i) {
        const long long row0 = e.y + quad * 32;
        const int rows = min(32, e.z - static_cast<int>(row0));  // of this warp; may be <= 0
        const int cols = (e.w & 3) * 64, n0 = (e.w >> 2) * 64;
        sums.zero();
        for (int k0 = 0; k0 < KS; k0 += chunk) {
          if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc.slot], acc.phase, abort_word, lim))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (rows > 0) sums.add(t_lane + acc.slot * 256, half, cols);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc.slot]);
          acc.advance();
        }
        if (!ok || rows <= 0) continue;
        if (E4M3)
          ok = fwd_rows_e4m3(args, stage, halves_of_rows, sums, half, lane, row0, rows, n0, units++, abort_word, lim);
        else
          fwd_rows_bf16(args, stage, sums, half, lane, row0, rows, n0, cols);
      }
    } else {
      for (uint32_t i = 0; queue.get(i, e, true, lane, abort_word, lim) && e.x >= 0; ++i) {
        const long long row0 = e.y + quad * 32;
        const int rows = min(32, e.z - static_cast<int>(row0));  // of this warp; may be <= 0
        const int cols = (e.w & 3) * 64;  // of this warp
        const int col0 = (e.w >> 2) * 128 + half * cols;
        // read while the products run
        Kept32<E4M3> kept;
        kept.fetch(args, row0, rows, col0, lane);
        float sa = 0.0f, sb = 0.0f;
        if (E4M3 && lane < rows) {
          sa = args.gus[(col0 / 128) * static_cast<long long>(args.M) + row0 + lane];
          sb = args.gus[(N / 128 + col0 / 128) * args.M + row0 + lane];
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc.slot], acc.phase, abort_word, lim))) break;
        tc_fence_after();
        if (rows > 0)
          bwd_rows<E4M3>(args, stage, t_lane + acc.slot * 256 + half * cols, lane, row0, rows, col0, cols, kept, sa, sb);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc.slot]);
        acc.advance();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
  if (threadIdx.x == 0) finish_claims(const_cast<int32_t*>(args.meta), *abort_word != 0);
}

template <bool FWD, bool E4M3>
cudaError_t launch(const CUtensorMap& map_a, const CUtensorMap& map_b, const SwigluArgs& args, int grid,
                   cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(gmm_swiglu_kernel<FWD, E4M3>, kSmemBytes, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(gmm_swiglu_kernel<FWD, E4M3>, dim3(grid), dim3(kThreads), kSmemBytes, stream, map_a, map_b, args);
}

}  // namespace

cudaError_t launch_gmm_swiglu_fwd(const CUtensorMap& map_x, const CUtensorMap& map_w, const SwigluArgs& args,
                                  int grid, cudaStream_t stream) {
  if (args.guq) return launch<true, true>(map_x, map_w, args, grid, stream);
  return launch<true, false>(map_x, map_w, args, grid, stream);
}

cudaError_t launch_gmm_swiglu_bwd(const CUtensorMap& map_dy, const CUtensorMap& map_w2, const SwigluArgs& args,
                                  int grid, cudaStream_t stream) {
  if (args.guq) return launch<false, true>(map_dy, map_w2, args, grid, stream);
  return launch<false, false>(map_dy, map_w2, args, grid, stream);
}

}  // namespace gmm
