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

// starts[b] = rows of the requests before b that have new tokens, at most the
// rows that there is room for.
__global__ void __launch_bounds__(kScanThreads)
    mla_expand_starts_kernel(const __grid_constant__ ChunkParams p, int32_t* starts, int32_t capacity) {
  __shared__ int64_t warp_sum[kScanThreads / 32];
  after_predecessor();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t each = (p.batch + kScanThreads - 1) / kScanThreads;
  const int32_t lo = min(static_cast<int32_t>(threadIdx.x) * each, p.batch), hi = min(lo + each, p.batch);
  int64_t sum = 0;
  for (int32_t b = lo; b < hi; ++b) {
    const ChunkRequest r(p, b);
    sum += r.count > 0 ? r.len : 0;
  }
  int64_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int64_t at = upto - sum;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  for (int32_t b = lo; b < hi; ++b) {
    starts[b] = static_cast<int32_t>(min(at, static_cast<int64_t>(capacity)));
    const ChunkRequest r(p, b);
    at += r.count > 0 ? r.len : 0;
  }
  if (threadIdx.x == kScanThreads - 1) starts[p.batch] = static_cast<int32_t>(min(at, static_cast<int64_t>(capacity)));
}

// One warp per kRowsOfWarp rows, whose slots its lanes find side by side.  Rows
// of pages outside the pool are left: whoever reads the table masks them.
template <int kKv>
__global__ void __launch_bounds__(32 * kWarps)
    mla_expand_kernel(const __grid_constant__ ChunkParams p, const int32_t* starts, uint16_t* rows) {
  after_predecessor();
  const int lane = threadIdx.x & 31;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kRowsOfWarp;
  const int64_t end = starts[p.batch];
  if (first >= end) return;
  int32_t slot = -1;
  if (lane < kRowsOfWarp && first + lane < end) {
    const int32_t row = static_cast<int32_t>(first) + lane;
    int32_t lo = 0, hi = p.batch - 1;   // the last request that starts at or before the row
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) / 2;
      if (starts[mid] <= row) lo = mid; else hi = mid - 1;
    }
    const int32_t t = row - starts[lo];
    const int32_t page = p.block_table[static_cast<int64_t>(lo) * p.max_pages + (t >> p.page_shift)];
    if (page >= 0 && page < p.num_pages) slot = (page << p.page_shift) + (t & ((1 << p.page_shift) - 1));
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
    if (at[i] < 0) continue;
    const RowWords r = cached_to_bf16(c[i], at[i]);
    uint16_t* out = rows + (first + i) * kDqk;
    reinterpret_cast<uint4*>(out)[lane] = r.a;
    reinterpret_cast<uint4*>(out)[32 + lane] = r.b;
    reinterpret_cast<uint32_t*>(out + kDc)[lane] = r.key;
  }
}

}  // namespace

cudaError_t launch_expand(const ChunkParams& p, const ChunkWorkspace& w, cudaStream_t stream) {
  const cudaError_t err = launch_dependent(mla_expand_starts_kernel, dim3(1), kScanThreads, 0, stream, p, w.starts, w.capacity);
  if (err != cudaSuccess || w.capacity == 0) return err;
  const dim3 blocks((w.capacity + kWarps * kRowsOfWarp - 1) / (kWarps * kRowsOfWarp));
  const auto launch = [&](auto kernel) {
    return launch_dependent(kernel, blocks, 32 * kWarps, 0, stream, p, static_cast<const int32_t*>(w.starts), w.rows);
  };
  return p.kv_dtype == MLA_KV_FP8_E4M3_E8M0 ? launch(mla_expand_kernel<MLA_KV_FP8_E4M3_E8M0>)
                                            : launch(mla_expand_kernel<MLA_KV_FP4_E2M1_E8M0>);
}

}  // namespace mla
