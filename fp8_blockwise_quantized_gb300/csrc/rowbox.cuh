// Row transposition of one warp through shared memory.  An epilogue thread
// works on one row (that is how tensor memory is read), but global memory
// wants whole 32-byte sectors and neighbouring lanes side by side: 16-byte
// stores of 32 lanes to 32 rows are half-sector writes, and cost the gated
// backward 120 of 280 us at 65536 rows.
#pragma once

#include <cstdint>

namespace gmm {

// 32 rows of ROWB bytes (32, 64 or 128) in 16-byte chunks; the chunk index is
// permuted within each 128 bytes so that neither a thread's row nor the
// lanes' sweep over rows meets a bank twice.
template <int ROWB>
struct RowBox {
  static constexpr int kBytes = 32 * ROWB;
  static constexpr int kChunks = ROWB / 16;       // per row
  static constexpr int kSweeps = kBytes / 512;    // warp-wide accesses that cover the box
  static constexpr int kRows = 32 / kChunks;      // rows per sweep
  static __device__ __forceinline__ uint4* at(uint8_t* box, int r, int j) {
    return reinterpret_cast<uint4*>(box + r * ROWB + ((j ^ ((r / (128 / ROWB)) & (kChunks - 1))) << 4));
  }
  // rows [0, nvalid) of global memory (row stride `ld` bytes) into registers,
  // lanes side by side; then into the box
  static __device__ __forceinline__ void fetch(uint4 (&v)[kSweeps], const uint8_t* g, long long ld, int nvalid,
                                               int lane) {
    const int j = lane % kChunks;
#pragma unroll
    for (int i = 0; i < kSweeps; ++i) {
      const int r = i * kRows + lane / kChunks;
      v[i] = r < nvalid ? __ldg(reinterpret_cast<const uint4*>(g + r * ld + 16 * j)) : make_uint4(0, 0, 0, 0);
    }
  }
  static __device__ __forceinline__ void put_sweeps(uint8_t* box, const uint4 (&v)[kSweeps], int lane) {
#pragma unroll
    for (int i = 0; i < kSweeps; ++i) *at(box, i * kRows + lane / kChunks, lane % kChunks) = v[i];
  }
  // this lane's row
  static __device__ __forceinline__ uint4 get(uint8_t* box, int lane, int j) { return *at(box, lane, j); }
  static __device__ __forceinline__ void put(uint8_t* box, int lane, int j, const uint4& v) { *at(box, lane, j) = v; }
  // rows [0, nvalid) of the box to global memory
  static __device__ __forceinline__ void store(uint8_t* box, uint8_t* g, long long ld, int nvalid, int lane) {
    const int j = lane % kChunks;
#pragma unroll
    for (int i = 0; i < kSweeps; ++i) {
      const int r = i * kRows + lane / kChunks;
      if (r < nvalid) *reinterpret_cast<uint4*>(g + r * ld + 16 * j) = *at(box, r, j);
    }
  }
};

}  // namespace gmm
