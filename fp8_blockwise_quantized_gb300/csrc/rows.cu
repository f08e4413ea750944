// Rows sorted by expert and joined again: the places of a batch's choices among
// the sorted rows, x's rows at their places, and the weighted sums back.
#include "common.cuh"
#include "kernels.cuh"
#include "metadata.cuh"
#include "mx4.cuh"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace gmm {

namespace {

// ---- places -------------------------------------------------------------------
// A stable counting sort of N ids into G + 1 bins, the last for the ids outside
// 0 .. G - 1.  A CTA takes a chunk of consecutive ids, each of its warps a run of
// the chunk, 32 ids a round; the warp's count of an id in the rounds before and the
// lanes before with the same id give its place in the run.  The lanes of one id find
// each other in a word of shared memory for each bin, or where there are too many bins
// for that by a ballot for each bit (65536 ids of 256: 6.2 us; by ballots 8.6; by the
// match instruction, which takes a round for each different id, 11.8).  The places'
// bases are the ids before in the chunk (summed over the warps), in the chunks before
// and in the bins before.  Up to 65536 ids the chunks are a cluster's CTAs, which read
// each other's counts; beyond, a first kernel leaves them in a table.
constexpr int kSortThreads = 512;
constexpr int kSortCluster = 8;
constexpr int kMaskBins = 1025;  // so many bins, and their words are at most 107 KB with the counts
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDirectChunks = 64;  // so many rows of the table each CTA sums itself

__device__ __forceinline__ int bin_of(int id, int G) {
  return static_cast<unsigned>(id) < static_cast<unsigned>(G) ? id : G;
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const int32_t* __restrict__ ids, int N, int G,
                                                                  int chunk, int32_t* __restrict__ table) {
  extern __shared__ int hist[];
  griddep_launch_dependents();
  const int B = G + 1;
  for (int b = threadIdx.x; b < B; b += kSortThreads) hist[b] = 0;
  __syncthreads();
  griddep_wait();  // the ids may come from the previous kernel
  const long long first = static_cast<long long>(blockIdx.x) * chunk;
  const int n = static_cast<int>(min(static_cast<long long>(chunk), N - first));
  for (int i = threadIdx.x; i < n; i += kSortThreads) atomicAdd(hist + bin_of(__ldg(ids + first + i), G), 1);
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += kSortThreads) table[static_cast<long long>(blockIdx.x) * B + b] = hist[b];
}

// Many chunks: the table's columns as sums of the rows before, and their totals behind the last row.
__global__ void __launch_bounds__(64) sort_scan_kernel(int32_t* __restrict__ table, int B, int chunks) {
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.x * 64 + threadIdx.x;
  if (b >= B) return;
  int run = 0;
  int32_t* p = table + b;
#pragma unroll 8
  for (int c = 0; c < chunks; ++c, p += B) {
    const int v = *p;
    *p = run;
    run += v;
  }
  *p = run;
}

// rounds: of a warp, at most R; a CTA's chunk is kSortThreads * rounds ids.
template <int R, bool CLUSTER, bool MASKS>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const int32_t* __restrict__ ids, int N, int G,
                                                                  int rounds, int chunks,
                                                                  const int32_t* __restrict__ table,
                                                                  int32_t* __restrict__ rows,
                                                                  int32_t* __restrict__ sizes) {
  extern __shared__ int smem[];
  __shared__ int warp_sums[kSortWarps];
  const int B = G + 1, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int* base = smem;                                           // [B]
  int* counts = smem + B;                                     // [B]
  uint16_t* runs = reinterpret_cast<uint16_t*>(smem + 2 * B);  // [kSortWarps][B]; a chunk has at most 8192 ids
  uint16_t* mine = runs + warp * B;
  griddep_launch_dependents();
  for (int b = t; b < kSortWarps / 2 * B; b += kSortThreads) reinterpret_cast<uint32_t*>(runs)[b] = 0;
  uint32_t* masks = reinterpret_cast<uint32_t*>(runs + kSortWarps * B);  // [kSortWarps][B]
  if constexpr (MASKS)
    for (int b = t; b < kSortWarps * B; b += kSortThreads) masks[b] = 0;
  const int bits = 32 - __clz(G);  // of a bin
  __syncthreads();
  griddep_wait();
  const long long first = (static_cast<long long>(blockIdx.x) * kSortThreads + warp * 32) * rounds + lane;
  int bin[R], rank[R];
#pragma unroll
  for (int r = 0; r < R; ++r) bin[r] = r < rounds && first + 32 * r < N ? bin_of(__ldg(ids + first + 32 * r), G) : -1;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r >= rounds) break;
    const bool live = bin[r] >= 0;  // the lanes behind the last id count nothing
    uint32_t* mask = masks + warp * B + bin[r];
    unsigned peers;
    if constexpr (MASKS) {
      if (live) atomicOr(mask, 1u << lane);
      __syncwarp();
      peers = live ? *mask : 0;
    } else {
      peers = __ballot_sync(0xffffffffu, live);
      for (int i = 0; i < bits; ++i) {
        const bool set = bin[r] >> i & 1;
        const unsigned with = __ballot_sync(0xffffffffu, set);
        peers &= set ? with : ~with;
      }
    }
    const int before = __popc(peers & ((1u << lane) - 1u));
    const int so_far = live ? mine[bin[r]] : 0;
    __syncwarp();
    if (live && before == 0) {
      mine[bin[r]] = static_cast<uint16_t>(so_far + __popc(peers));
      if constexpr (MASKS) *mask = 0;
    }
    __syncwarp();
    rank[r] = so_far + before;
  }
  __syncthreads();
  // per bin: the warps' counts as sums of those before, the chunks before, all chunks
  const int per = (B + kSortThreads - 1) / kSortThreads, b0 = min(B, t * per), b1 = min(B, b0 + per);
  for (int b = b0; b < b1; ++b) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = runs[w * B + b];
      runs[w * B + b] = static_cast<uint16_t>(run);
      run += c;
    }
    counts[b] = run;
  }
  if constexpr (CLUSTER) {
    __syncwarp();
    cluster_sync_all();
  }
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    int earlier = 0, total = counts[b];
    if constexpr (CLUSTER) {
      total = 0;
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c) {
        int v;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(counts + b), c)));
        if (c < static_cast<int>(blockIdx.x)) earlier += v;
        total += v;
      }
    } else if (chunks > kDirectChunks) {
      earlier = table[static_cast<long long>(blockIdx.x) * B + b];
      total = table[static_cast<long long>(chunks) * B + b];
    } else if (chunks > 1) {
      total = 0;
#pragma unroll 8
      for (int c = 0; c < chunks; ++c) {
        const int v = table[c * B + b];
        if (c < static_cast<int>(blockIdx.x)) earlier += v;
        total += v;
      }
    }
    if (blockIdx.x == 0 && b < G) sizes[b] = total;
    base[b] = sum + earlier;
    sum += total;
  }
  const int inc = warp_inclusive_scan(sum);
  if (lane == 31) warp_sums[warp] = inc;
  // (the other CTAs' counts have been read: none of them leaves before)
  if constexpr (CLUSTER) {
    __syncwarp();
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  int start = inc - sum;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) start += w < warp ? warp_sums[w] : 0;
  for (int b = b0; b < b1; ++b) base[b] += start;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r >= rounds || bin[r] < 0) continue;
    const int row = base[bin[r]] + mine[bin[r]] + rank[r];
    rows[first + 32 * r] = bin[r] < G ? row : -1 - row;
  }
}

// ---- x by token -> sorted rows --------------------------------------------------
// The place of a choice, or -1 where rows holds what no sort gives.
__device__ __forceinline__ long long place_of(int row, long long M) {
  const long long p = row >= 0 ? row : -1LL - row;
  return p < M ? p : -1;
}

// A thread takes 8 values of a token and writes them to the token's k places.
template <typename I>
__global__ void __launch_bounds__(256) gather_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ rows,
                                                     I vectors, int k, unsigned KV, long long M,
                                                     uint4* __restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  const I v = static_cast<I>(blockIdx.x) * 256 + threadIdx.x;
  if (v >= vectors) return;
  const I t = v / KV;
  const unsigned c = static_cast<unsigned>(v - t * KV);
  const uint4 val = __ldcs(x + v);
  const int32_t* at = rows + static_cast<long long>(t) * k;
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int row = __ldg(at + j);
    const long long p = place_of(row, M);
    if (p >= 0) out[p * KV + c] = row >= 0 ? val : make_uint4(0, 0, 0, 0);
  }
}

// The same with the 1x128 e4m3 quantisation of gmm_quantize_lhs in between: each
// token is quantised once, whatever its number of places.  Eight lanes take a
// block of 128 values.  8192 tokens of 8 choices, 2048 columns: 29.5 us (floor 25.8);
// what it has beyond the floor are the scales, 4 bytes a sector here and there.
template <typename I>
__global__ void __launch_bounds__(256) gather_quantize_kernel(const uint4* __restrict__ x,
                                                              const int32_t* __restrict__ rows, I units, int k,
                                                              unsigned KB, long long M, uint4* __restrict__ xq,
                                                              float* __restrict__ xs) {
  griddep_launch_dependents();
  griddep_wait();
  const I v = static_cast<I>(blockIdx.x) * 256 + threadIdx.x;
  const I u = v >> 3;
  const unsigned l8 = threadIdx.x & 7;
  const bool live = u < units;
  const I t = u / KB;
  const unsigned kb = static_cast<unsigned>(u - t * KB);
  uint4 a = make_uint4(0, 0, 0, 0), b = a;
  const int32_t* at = rows + static_cast<long long>(t) * k;
  // a token that no expert has is not read; the first eight places are kept
  int first[8];
  bool any = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    first[j] = live && j < k ? __ldg(at + j) : INT32_MIN;
    any |= first[j] >= 0;
  }
  if (live)
    for (int j = 8; j < k; ++j) any |= __ldg(at + j) >= 0;
  if (any) {
    a = __ldcs(x + 2 * static_cast<long long>(v));
    b = __ldcs(x + 2 * static_cast<long long>(v) + 1);
  }
  float m = fmaxf(bf16x8_absmax(a), bf16x8_absmax(b));
#pragma unroll
  for (int d = 4; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (!live) return;
  float s, inv;
  e4m3_block_scale(m, s, inv);
  const uint2 qa = bf16x8_to_e4m3(a, inv), qb = bf16x8_to_e4m3(b, inv);
  const uint4 q = make_uint4(qa.x, qa.y, qb.x, qb.y);
  auto send = [&](int row, int j) {
    const long long p = place_of(row, M);
    if (p < 0) return;
    xq[(p * KB + kb) * 8 + l8] = row >= 0 ? q : make_uint4(0, 0, 0, 0);
    if (j >= 8 && l8 == (j & 7)) xs[kb * M + p] = row >= 0 ? s : 0.0f;
  };
  int own = first[0];  // each of the eight lanes writes one choice's scale
#pragma unroll
  for (int j = 1; j < 8; ++j)
    if (l8 == j) own = first[j];
  const long long po = place_of(own, M);
  if (po >= 0) xs[kb * M + po] = own >= 0 ? s : 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= k) break;
    send(first[j], j);
  }
  for (int j = 8; j < k; ++j) send(__ldg(at + j), j);
}

// And with the MXFP4 quantisation of gmm_mx4_quantize_lhs: a lane's 16 values are half
// of a block of 32, the four scale bytes of 128 columns one word.  8192 tokens of 8
// choices, 2048 columns: 20.0 us (floor 15.7; gather, then quantiser 94), the rest the
// scales as above.
template <typename I>
__global__ void __launch_bounds__(256) gather_mx4_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ rows,
                                                         I units, int k, unsigned KB, long long M,
                                                         uint2* __restrict__ xq, uint32_t* __restrict__ xs) {
  griddep_launch_dependents();
  griddep_wait();
  const I v = static_cast<I>(blockIdx.x) * 256 + threadIdx.x;
  const I u = v >> 3;
  const unsigned l8 = threadIdx.x & 7, lane = threadIdx.x & 31;
  const bool live = u < units;
  const I t = u / KB;
  const unsigned kb = static_cast<unsigned>(u - t * KB);
  const int32_t* at = rows + static_cast<long long>(t) * k;
  bool any = false;  // as in gather_quantize_kernel
  if (live)
    for (int j = 0; j < k; ++j) any |= __ldg(at + j) >= 0;
  uint4 a = make_uint4(0, 0, 0, 0), b = a;
  if (any) {
    a = __ldcs(x + 2 * static_cast<long long>(v));
    b = __ldcs(x + 2 * static_cast<long long>(v) + 1);
  }
  const uint32_t pa[4] = {a.x, a.y, a.z, a.w}, pb[4] = {b.x, b.y, b.z, b.w};
  uint32_t m2 = absmax2(absmax2(absmax2(pa[0], pa[1]), absmax2(pa[2], pa[3])),
                        absmax2(absmax2(pb[0], pb[1]), absmax2(pb[2], pb[3])));
  m2 = absmax2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
  m2 = absmax2(m2, m2 >> 16);
  const uint32_t byte = mx4_scale_byte(m2 & 0xffffu), inv = mx4_inverse2(byte);
  const uint2 q = make_uint2(mx4_codes8(pa, inv), mx4_codes8(pb, inv));
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) word |= __shfl_sync(0xffffffffu, byte, (lane & 24u) + 2 * i) << (8 * i);
  if (!live) return;
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int row = __ldg(at + j);
    const long long p = place_of(row, M);
    if (p < 0) continue;
    xq[(p * KB + kb) * 8 + l8] = row >= 0 ? q : make_uint2(0, 0);
    if (l8 == (j & 7)) xs[kb * M + p] = row >= 0 ? word : 0u;
  }
}

// ---- sorted rows -> tokens --------------------------------------------------------
// A thread sums V vectors of 8 columns of a token over its choices, in their order:
// one, with four choices' loads on their way at once, or two of two choices (16384
// tokens of 2 choices, 4096 columns: 75.6 -> 64.7 us).  8192 tokens of 8 choices,
// 2048 columns: 45.3 us, the floor.
template <typename I, int V>
__global__ void __launch_bounds__(256) combine_kernel(const uint4* __restrict__ y, const int32_t* __restrict__ rows,
                                                      const float* __restrict__ weights, I units, int k, unsigned KV,
                                                      unsigned part, long long M, uint4* __restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  const I u = static_cast<I>(blockIdx.x) * 256 + threadIdx.x;
  if (u >= units) return;
  const I t = u / part;
  const unsigned c = static_cast<unsigned>(u - t * part);
  const long long e0 = static_cast<long long>(t) * k;
  float acc[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v][i] = 0.0f;
  for (int j0 = 0; j0 < k; j0 += 4 / V) {
    uint4 val[4 / V][V];
    float w[4 / V];
#pragma unroll
    for (int j = 0; j < 4 / V; ++j) {
      const int row = j0 + j < k ? __ldg(rows + e0 + j0 + j) : -1;
      const bool live = row >= 0 && row < M;
      w[j] = live ? (weights ? __ldg(weights + e0 + j0 + j) : 1.0f) : 0.0f;
      // a row of no group adds nothing, whatever its weight holds
#pragma unroll
      for (int v = 0; v < V; ++v)
        val[j][v] = live && c + v * part < KV ? __ldcs(y + static_cast<long long>(row) * KV + c + v * part)
                                              : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 4 / V; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f[8];
        unpack8(val[j][v], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[v][i] = fmaf(w[j], f[i], acc[v][i]);
      }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (c + v * part < KV) out[static_cast<long long>(t) * KV + c + v * part] = pack8(acc[v]);
}

// The gradient: dy = weight * dout at each place (zero at those of no group), and
// the weight's gradient, the product of dout's row and y's.  A group of `span`
// warps takes a token, so that the products' sums stay in registers; dout's row is
// read for four choices at a time (of eight, the registers leave room for two CTAs an
// SM in place of four: 1024 tokens of 8 choices, 2048 columns, 14.1 us for 11.4, floor
// 10.5; 8192 tokens 97.0 for 93.1, floor 85.6).
constexpr int kBwdWarps = 8, kBwdChoices = 4;
__global__ void __launch_bounds__(32 * kBwdWarps, 4) combine_bwd_kernel(const uint4* __restrict__ dout,
                                                                     const uint4* __restrict__ y,
                                                                     const int32_t* __restrict__ rows,
                                                                     const float* __restrict__ weights, long long T,
                                                                     int k, unsigned KV, int span,
                                                                     uint4* __restrict__ dy,
                                                                     float* __restrict__ dweights) {
  __shared__ float part[kBwdWarps][kBwdChoices];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / span, in = warp - team * span;
  const long long t = static_cast<long long>(blockIdx.x) * (kBwdWarps / span) + team, M = T * k;
  const long long e0 = t * k;
  for (int j0 = 0; j0 < k; j0 += kBwdChoices) {
    const int many = min(kBwdChoices, k - j0);
    float dot[kBwdChoices], w[kBwdChoices];
    int row[kBwdChoices];
#pragma unroll
    for (int j = 0; j < kBwdChoices; ++j) {
      dot[j] = w[j] = 0.0f;
      row[j] = INT32_MIN;
      if (t < T && j < many) {
        row[j] = __ldg(rows + e0 + j0 + j);
        w[j] = row[j] >= 0 ? __ldg(weights + e0 + j0 + j) : 0.0f;
      }
    }
    if (t < T) {
      for (unsigned c = in * 32 + lane; c < KV; c += span * 32) {
        float d[8];
        unpack8(__ldg(dout + t * KV + c), d);
        uint4 val[kBwdChoices];
#pragma unroll
        for (int j = 0; j < kBwdChoices; ++j)
          val[j] = row[j] >= 0 && row[j] < M ? __ldcs(y + static_cast<long long>(row[j]) * KV + c)
                                             : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < kBwdChoices; ++j) {
          if (j >= many) break;
          float f[8], o[8];
          unpack8(val[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = fmaf(d[i], f[i], dot[j]);
            o[i] = w[j] * d[i];
          }
          const long long p = place_of(row[j], M);
          if (p >= 0) dy[p * KV + c] = row[j] >= 0 ? pack8(o) : make_uint4(0, 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kBwdChoices; ++j) dot[j] = warp_sum(dot[j]);
    if (span > 1) {
      __syncthreads();  // the previous choices' sums have been read
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < kBwdChoices; ++j) part[warp][j] = dot[j];
      }
      __syncthreads();
      if (in == 0) {
#pragma unroll
        for (int j = 0; j < kBwdChoices; ++j)
          for (int s = 1; s < span; ++s) dot[j] += part[warp + s][j];
      }
    }
    if (t < T && in == 0) {
#pragma unroll
      for (int j = 0; j < kBwdChoices; ++j)
        if (lane == j && j < many) dweights[e0 + j0 + j] = row[j] >= 0 ? dot[j] : 0.0f;
    }
  }
}

constexpr long long kNarrow = 1LL << 31;  // indices below it are 32 bits

unsigned blocks_of(long long threads) { return static_cast<unsigned>((threads + 255) / 256); }

constexpr int64_t kOneCta = 2048, kOneCluster = kSortCluster * kSortThreads * 16;
// Rounds of a warp in a table's sort: few while that gives chunks for a good part of the SMs.
int sort_rounds(int64_t N) { return N <= 131072 ? 4 : 16; }
// chunks of a table's sort; 1 where a CTA or a cluster holds all ids
int sort_chunks(int64_t N) {
  const int64_t chunk = kSortThreads * sort_rounds(N);
  return N <= kOneCluster ? 1 : static_cast<int>((N + chunk - 1) / chunk);
}

}  // namespace

size_t sort_scratch_bytes(int64_t N, int G) {
  const int chunks = sort_chunks(N);
  return chunks > 1 ? static_cast<size_t>(chunks + 1) * (G + 1) * sizeof(int32_t) : 0;
}

cudaError_t launch_sort_rows(const int32_t* ids, int64_t N, int G, int32_t* rows, int32_t* sizes, void* scratch,
                             cudaStream_t stream) {
  const int B = G + 1, n = static_cast<int>(N), chunks = sort_chunks(N);
  int32_t* table = static_cast<int32_t*>(scratch);
  // 16384 ids sort in the time of those 32 MB
  const bool over = launch_over(2048LL * N, stream);
  cudaError_t e;
  if (chunks > 1) {
    e = launch_pdl(sort_count_kernel, dim3(chunks), dim3(kSortThreads), B * sizeof(int), stream, ids, n, G,
                   kSortThreads * sort_rounds(N), table);
    if (e != cudaSuccess) return e;
    if (chunks > kDirectChunks &&
        (e = launch_pdl(sort_scan_kernel, dim3((B + 63) / 64), dim3(64), 0, stream, table, B, chunks)) != cudaSuccess)
      return e;
  }
  const bool cluster = N > kOneCta && N <= kOneCluster;
  const int ctas = cluster ? kSortCluster : chunks;
  const int rounds =
      chunks > 1 ? sort_rounds(N) : static_cast<int>((N + ctas * kSortThreads - 1) / (ctas * kSortThreads));
  static std::atomic<uint64_t> done[2][5];
  auto place = [&](auto masks, auto kernel, int i) {
    constexpr bool kMasks = decltype(masks)::value;
    const auto bytes = [](int bins) { return bins * (2 * 4 + kSortWarps * (kMasks ? 6 : 2)); };
    if (bytes(B) > 40 * 1024) {
      const cudaError_t err = allow_smem(kernel, bytes(kMasks ? kMaskBins : kMaxGroups + 1), done[kMasks][i]);
      if (err != cudaSuccess) return err;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = bytes(B);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int attrs = 0;
    if (cluster) {
      attr[attrs].id = cudaLaunchAttributeClusterDimension;
      attr[attrs].val.clusterDim.x = kSortCluster;
      attr[attrs].val.clusterDim.y = attr[attrs].val.clusterDim.z = 1;
      ++attrs;
    }
    if (over) {
      attr[attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[attrs].val.programmaticStreamSerializationAllowed = 1;
      ++attrs;
    }
    cfg.attrs = attr;
    cfg.numAttrs = attrs;
    return cudaLaunchKernelEx(&cfg, kernel, ids, n, G, rounds, chunks, static_cast<const int32_t*>(table), rows, sizes);
  };
  auto sized = [&](auto masks) {
    constexpr bool M = decltype(masks)::value;
    if (cluster)
      return rounds <= 4 ? place(masks, sort_place_kernel<4, true, M>, 0)
                         : place(masks, sort_place_kernel<16, true, M>, 1);
    if (rounds <= 1) return place(masks, sort_place_kernel<1, false, M>, 2);
    return rounds <= 4 ? place(masks, sort_place_kernel<4, false, M>, 3)
                       : place(masks, sort_place_kernel<16, false, M>, 4);
  };
  return B <= kMaskBins ? sized(std::true_type()) : sized(std::false_type());
}

cudaError_t launch_gather_rows(const void* x, const int32_t* rows, int64_t T, int k, int64_t K, void* out,
                               cudaStream_t stream) {
  const long long vectors = T * (K / 8), M = T * k;
  const unsigned KV = static_cast<unsigned>(K / 8);
  const bool over = launch_over(2 * M * K, stream);
  if (vectors < kNarrow)
    return launch_short(over, gather_kernel<uint32_t>, dim3(blocks_of(vectors)), dim3(256), 0, stream,
                        static_cast<const uint4*>(x), rows, static_cast<uint32_t>(vectors), k, KV, M,
                        static_cast<uint4*>(out));
  return launch_short(over, gather_kernel<uint64_t>, dim3(blocks_of(vectors)), dim3(256), 0, stream,
                      static_cast<const uint4*>(x), rows, static_cast<uint64_t>(vectors), k, KV, M,
                      static_cast<uint4*>(out));
}

cudaError_t launch_gather_quantize(const void* x, const int32_t* rows, int64_t T, int k, int64_t K, void* xq, float* xs,
                                   cudaStream_t stream) {
  const long long units = T * (K / 128), M = T * k;
  const unsigned KB = static_cast<unsigned>(K / 128);
  const bool over = launch_over(M * K, stream);
  if (units < kNarrow / 8)
    return launch_short(over, gather_quantize_kernel<uint32_t>, dim3(blocks_of(units * 8)), dim3(256), 0, stream,
                        static_cast<const uint4*>(x), rows, static_cast<uint32_t>(units), k, KB, M,
                        static_cast<uint4*>(xq), xs);
  return launch_short(over, gather_quantize_kernel<uint64_t>, dim3(blocks_of(units * 8)), dim3(256), 0, stream,
                      static_cast<const uint4*>(x), rows, static_cast<uint64_t>(units), k, KB, M,
                      static_cast<uint4*>(xq), xs);
}

cudaError_t launch_gather_mx4(const void* x, const int32_t* rows, int64_t T, int k, int64_t K, void* xq, void* xs,
                              cudaStream_t stream) {
  const long long units = T * (K / 128), M = T * k;
  const unsigned KB = static_cast<unsigned>(K / 128);
  const bool over = launch_over(M * K / 2, stream);
  if (units < kNarrow / 8)
    return launch_short(over, gather_mx4_kernel<uint32_t>, dim3(blocks_of(units * 8)), dim3(256), 0, stream,
                        static_cast<const uint4*>(x), rows, static_cast<uint32_t>(units), k, KB, M,
                        static_cast<uint2*>(xq), static_cast<uint32_t*>(xs));
  return launch_short(over, gather_mx4_kernel<uint64_t>, dim3(blocks_of(units * 8)), dim3(256), 0, stream,
                      static_cast<const uint4*>(x), rows, static_cast<uint64_t>(units), k, KB, M,
                      static_cast<uint2*>(xq), static_cast<uint32_t*>(xs));
}

cudaError_t launch_combine_rows(const void* y, const int32_t* rows, const float* weights, int64_t T, int k, int64_t K,
                                void* out, cudaStream_t stream) {
  const unsigned KV = static_cast<unsigned>(K / 8);
  const int V = k <= 2 ? 2 : 1;
  const unsigned part = (KV + V - 1) / V;
  const long long units = T * static_cast<long long>(part), M = T * k;
  const bool over = launch_over(2 * M * K, stream);
  auto launch = [&](auto kernel, auto narrow) {
    return launch_short(over, kernel, dim3(blocks_of(units)), dim3(256), 0, stream, static_cast<const uint4*>(y), rows,
                        weights, static_cast<decltype(narrow)>(units), k, KV, part, M, static_cast<uint4*>(out));
  };
  if (units < kNarrow)
    return V == 2 ? launch(combine_kernel<uint32_t, 2>, uint32_t()) : launch(combine_kernel<uint32_t, 1>, uint32_t());
  return V == 2 ? launch(combine_kernel<uint64_t, 2>, uint64_t()) : launch(combine_kernel<uint64_t, 1>, uint64_t());
}

cudaError_t launch_combine_rows_bwd(const void* dout, const void* y, const int32_t* rows, const float* weights,
                                    int64_t T, int k, int64_t K, void* dy, float* dweights, int sms,
                                    cudaStream_t stream) {
  // a warp a token once that gives every SM 16 warps; more of them for few tokens
  int span = 1;
  while (span < kBwdWarps && T * span < 16LL * sms && span * 256 < K) span *= 2;
  const long long per = kBwdWarps / span;
  const bool over = launch_over(4 * T * k * K, stream);
  return launch_short(over, combine_bwd_kernel, dim3(static_cast<unsigned>((T + per - 1) / per)), dim3(32 * kBwdWarps),
                      0, stream, static_cast<const uint4*>(dout), static_cast<const uint4*>(y), rows, weights,
                      static_cast<long long>(T), k, static_cast<unsigned>(K / 8), span, static_cast<uint4*>(dy),
                      dweights);
}

}  // namespace gmm
