// A quantised cache's rows as bf16 rows in a workspace, one request behind the
// other, for operators that read each row many times: every code is converted
// once instead of once for each tile of queries.
#include <cuda_runtime.h>

#include "mla_chunk_internal.h"
#include "mla_rows.cuh"

namespace mla {

namespace {

constexpr int kScanThreads = 256;
constexpr int kWarps = 4, kRowsOfWarp = 4;
// Blocks a multiprocessor.  The grid is that of the plan's room, what there is of rows
// is known on the device alone: up to kBlocksOnce a block for every 16 rows of the room,
// beyond it kBlocksLoop whose warps go on to further rows.  294,912 rows in a room of
// as many (121 blocks): the weights of a decode step from FP8 152 us, looping 155;
// 25,534 rows in a room of 8,388,608: 24.7 us, with a block for every 16 546.
constexpr int kBlocksOnce = 128, kBlocksLoop = 32;
static_assert(kDensePad % kRowsOfWarp == 0, "a warp's rows are all there or none");

// Sum over the block's threads before this one, and the block's.
__device__ __forceinline__ int64_t sum_before(int64_t* warp_sum, int64_t v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int64_t at = upto - v;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  __syncthreads();
  return at;
}

// Each request's first expanded row and rows: of those that have new tokens, in
// order, as many as there is room for.
__global__ void __launch_bounds__(kScanThreads)
    mla_expand_starts_kernel(const __grid_constant__ ChunkParams p, int2* starts, int32_t context) {
  __shared__ int64_t warp_sum[kScanThreads / 32];
  after_predecessor();
  const int32_t each = (p.batch + kScanThreads - 1) / kScanThreads;
  const int32_t lo = min(static_cast<int32_t>(threadIdx.x) * each, p.batch), hi = min(lo + each, p.batch);
  const auto rows_of = [&](int32_t b) {
    const ChunkRequest r(p, b);
    return r.count > 0 ? r.len : 0;
  };
  int64_t sum = 0;
  for (int32_t b = lo; b < hi; ++b) sum += rows_of(b);
  const int64_t before = sum_before(warp_sum, sum);
  const auto there_of = [&](int32_t rows, int64_t at) {
    return static_cast<int32_t>(min(static_cast<int64_t>(rows), max(context - at, int64_t{0})));
  };
  const auto padded = [](int32_t rows) { return (static_cast<int64_t>(rows) + kDensePad - 1) / kDensePad * kDensePad; };
  int64_t at = before;
  sum = 0;
  for (int32_t b = lo; b < hi; ++b) {
    const int32_t rows = rows_of(b);
    sum += padded(there_of(rows, at));
    at += rows;
  }
  int64_t first = sum_before(warp_sum, sum);
  at = before;
  for (int32_t b = lo; b < hi; ++b) {
    const int32_t rows = rows_of(b), there = there_of(rows, at);
    starts[b] = make_int2(static_cast<int32_t>(first), there);
    first += padded(there);
    at += rows;
  }
  if (threadIdx.x == kScanThreads - 1) starts[p.batch] = make_int2(static_cast<int32_t>(first), 0);
}

// One warp per kRowsOfWarp rows, whose slots its lanes find side by side.  Padding,
// and rows of pages outside the pool, are zeros.  Bound by memory: 67,200 rows out of
// FP8 and 77 MB written in 18 us.
template <int kKv, bool kLoop>
__global__ void __launch_bounds__(32 * kWarps)
    mla_expand_kernel(const __grid_constant__ ChunkParams p, const int2* starts, uint16_t* rows) {
  after_predecessor();
  const int lane = threadIdx.x & 31;
  const uint32_t end = starts[p.batch].x;   // a multiple of kRowsOfWarp, as kDensePad is
#pragma unroll 1
  for (uint32_t first = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRowsOfWarp; first < end;
       first = kLoop ? first + gridDim.x * (kWarps * kRowsOfWarp) : end) {
    int32_t slot = -1;
    if (lane < kRowsOfWarp) {
      const int32_t row = static_cast<int32_t>(first) + lane;
      int32_t lo = 0, hi = p.batch - 1;   // the last request that starts at or before the row
      while (lo < hi) {
        const int32_t mid = (lo + hi + 1) / 2;
        if (starts[mid].x <= row) lo = mid; else hi = mid - 1;
      }
      const int2 at = starts[lo];
      const int32_t t = row - at.x;
      if (t < at.y) {
        const int32_t page = p.block_table[static_cast<int64_t>(lo) * p.max_pages + (t >> p.page_shift)];
        if (page >= 0 && page < p.num_pages) slot = (page << p.page_shift) + (t & ((1 << p.page_shift) - 1));
      }
    }
    CachedRow<kKv> c[kRowsOfWarp];
    int32_t at[kRowsOfWarp];
#pragma unroll
    for (int i = 0; i < kRowsOfWarp; ++i) {
      at[i] = __shfl_sync(0xffffffffu, slot, i);
      if (at[i] >= 0) load_cached(&c[i], p.kv, at[i], lane);
    }
#pragma unroll
    for (int i = 0; i < kRowsOfWarp; ++i) {
      RowWords r = {};
      if (at[i] >= 0) r = cached_to_bf16(c[i], at[i]);
      uint16_t* out = rows + static_cast<int64_t>(first + i) * kDqk;
      reinterpret_cast<uint4*>(out)[lane] = r.a;
      reinterpret_cast<uint4*>(out)[32 + lane] = r.b;
      reinterpret_cast<uint32_t*>(out + kDc)[lane] = r.key;
    }
  }
}

}  // namespace

cudaError_t launch_expand(const ChunkParams& p, const ChunkWorkspace& w, cudaStream_t stream) {
  const cudaError_t err = launch_dependent(mla_expand_starts_kernel, dim3(1), kScanThreads, 0, stream, p, w.starts, w.context);
  if (err != cudaSuccess || w.context == 0) return err;
  const int64_t units = (static_cast<int64_t>(w.capacity) + kWarps * kRowsOfWarp - 1) / (kWarps * kRowsOfWarp);
  const int64_t sms = 2 * w.clusters;
  const bool loop = units > kBlocksOnce * sms;
  const dim3 blocks(static_cast<unsigned>(loop ? kBlocksLoop * sms : units));
  const auto launch = [&](auto kernel) {
    return launch_dependent(kernel, blocks, 32 * kWarps, 0, stream, p, static_cast<const int2*>(w.starts), w.rows);
  };
  return p.kv_dtype == MLA_KV_FP8_E4M3_E8M0
             ? launch(loop ? mla_expand_kernel<MLA_KV_FP8_E4M3_E8M0, true> : mla_expand_kernel<MLA_KV_FP8_E4M3_E8M0, false>)
             : launch(loop ? mla_expand_kernel<MLA_KV_FP4_E2M1_E8M0, true> : mla_expand_kernel<MLA_KV_FP4_E2M1_E8M0, false>);
}

}  // namespace mla
