// What the kernels over pairs of CTAs (chunk attention, cached rows' weights) share:
// where a tile's cached rows are, and bounded waits.
#pragma once

#include "mla_chunk_internal.h"
#include "mla_pair.cuh"

namespace mla {

constexpr int kTileRows = 128;          // cached rows of a tile
constexpr uint64_t kWaitLimitNs = 1000000000ull;   // 1 s per wait

// 2^x with the hardware approximation (2^-22 relative; 2^-inf = 0), in bf16 weights and
// in sums that one thread adds in 32 bits.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Rows of a request that there are, from where on they are masked out.  dense: as in
// ChunkWorkspace::starts, null where rows are read in pages.
__device__ __forceinline__ int32_t rows_there(const int2* dense, const ChunkRequest& r, int32_t b) {
  return dense && r.count > 0 ? dense[b].y : r.len;
}

// The pages of a tile, looked up a tile ahead: lane l < 8 has the one of the tile's
// tokens 16 l .. 16 l + 15.
struct TilePages {
  int32_t page;
  __device__ __forceinline__ void load(const ChunkParams& c, int32_t b, int32_t limit, int32_t tile, int lane) {
    const int64_t tok = static_cast<int64_t>(tile) * kTileRows + 16 * (lane & 7);
    page = tok < limit ? c.block_table[static_cast<int64_t>(b) * c.max_pages + (tok >> c.page_shift)] : 0;
  }
  // pieces of 16 tokens in pages outside the pool
  __device__ __forceinline__ uint32_t bad(const ChunkParams& c) const {
    return __ballot_sync(0xffffffffu, page < 0 || page >= c.num_pages) & 255u;
  }
};

// Where a tile's cached rows are: lane l < 8 holds the pool row of the tile's
// tokens 16 l .. 16 l + 15, or -1.
struct TileRows {
  int32_t base, left;           // left: rows of the request from the tile's first on
  // dense: the request's first expanded row, or -1 where rows are in pages.  An
  // expanded request ends with zeros to a multiple of kDensePad rows, and those of
  // pages that are not there are zeros.
  __device__ __forceinline__ TileRows(const ChunkParams& c, int32_t limit, int32_t tile, const TilePages& at,
                                      int32_t dense, int lane) {
    const int64_t first = static_cast<int64_t>(tile) * kTileRows;
    const int32_t in = 16 * (lane & 7);
    left = static_cast<int32_t>(max(static_cast<int64_t>(limit) - first, int64_t{0}));
    base = -1;
    if (dense >= 0) {
      left = (left + kDensePad - 1) / kDensePad * kDensePad;
      if (in < left) base = dense + static_cast<int32_t>(first) + in;
    } else if (in < left && at.page >= 0 && at.page < c.num_pages) {
      base = (at.page << c.page_shift) + ((static_cast<int32_t>(first) + in) & ((1 << c.page_shift) - 1));
    }
  }
  // the pool rows of four tokens from t (of the tile, a multiple of 4), -1 for none
  __device__ __forceinline__ void four(int32_t t, int32_t (&row)[4]) const {
    const int32_t at = __shfl_sync(0xffffffffu, base, t >> 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) row[q] = at >= 0 && t + q < left ? at + (t & 15) + q : -1;
  }
};

// A wait of a role; false once a role of this CTA has given up (*abort).  What rarely
// runs is kept out of the loops around it: the roles' loops run from the
// instruction cache, and every one of them runs its own.
static __device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, int* abort, uint32_t* status) {
  if (pair_wait(bar, parity, abort, kWaitLimitNs)) return true;
  *static_cast<volatile int*>(abort) = 1;
  if (status) atomicOr(status, MLA_STATUS_TIMEOUT);
  return false;
}

// Copies in flight when a role has given up land within microseconds.
static __device__ __noinline__ void let_copies_land() {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
}

}  // namespace mla
