// The weights that queries give to cached rows: one warp per cached row.
#include <cuda_runtime.h>

#include "mla_chunk_internal.h"
#include "mla_rows.cuh"

namespace mla {

namespace {

constexpr int kWarps = 8;

struct RowValues {   // a lane's 18 of a row's 576 values
  float v[18];
};

__device__ __forceinline__ RowValues values_of(const RowWords& r) {
  RowValues x;
  const uint32_t w[9] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w, r.key};
#pragma unroll
  for (int i = 0; i < 9; ++i) {
    x.v[2 * i] = bf16_lo(w[i]);
    x.v[2 * i + 1] = bf16_hi(w[i]);
  }
  return x;
}

__device__ __forceinline__ float dot(const RowValues& a, const RowValues& b) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 18; ++i) s = fmaf(a.v[i], b.v[i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// The pool slot of row t of request b, or -1.
__device__ __forceinline__ int32_t slot_of(const ChunkParams& p, int32_t b, int32_t t) {
  const int32_t page = p.block_table[static_cast<int64_t>(b) * p.max_pages + (t >> p.page_shift)];
  if (page < 0 || page >= p.num_pages) {
    if (p.status) atomicOr(p.status, MLA_STATUS_BAD_PAGE);
    return -1;
  }
  return (page << p.page_shift) + (t & ((1 << p.page_shift) - 1));
}

template <int kKv>
__device__ __forceinline__ RowValues cached_row(const ChunkParams& p, int32_t slot, int lane) {
  CachedRow<kKv> c;
  load_cached(&c, p.kv, slot, lane);
  return values_of(cached_to_bf16(c, slot));
}

template <int kKv>
__global__ void __launch_bounds__(32 * kWarps) mla_cache_weights_kernel(const __grid_constant__ WeightsParams p) {
  const int lane = threadIdx.x & 31;
  after_predecessor();
  const int32_t b = blockIdx.y;
  const ChunkRequest r(p.c, b);
  if (r.bad && p.c.status && threadIdx.x == 0) atomicOr(p.c.status, MLA_STATUS_BAD_INDEX);
  const int64_t end = r.len < p.stride ? r.len : p.stride;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < end;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    float sum = 0.f;
    const int32_t slot = r.count > 0 ? slot_of(p.c, b, static_cast<int32_t>(t)) : -1;
    if (slot >= 0) {
      const RowValues k = cached_row<kKv>(p.c, slot, lane);
      for (int32_t j = 0; j < r.count; ++j) {
        if (t >= r.seen(j, p.c.causal)) continue;
        for (int32_t h = 0; h < p.c.heads; ++h) {
          const int64_t row = static_cast<int64_t>(r.first + j) * p.c.heads + h;
          RowWords qw;
          load_row(&qw, p.c.q + row * kDqk, lane);
          const float lse = p.lse[row];
          const float s = dot(values_of(qw), k) * p.c.scale_log2;
          sum += lse == -INFINITY ? 0.f : exp2f(s - lse * 1.4426950408889634f);
        }
      }
    }
    if (lane == 0) p.out[b * p.stride + t] = (p.in ? p.in[b * p.stride + t] : 0.f) + sum;
  }
}

}  // namespace

cudaError_t launch_cache_weights(const WeightsParams& p, cudaStream_t stream) {
  const dim3 grid(1024, p.c.batch);
  const auto launch = [&](auto kernel) { return launch_dependent(kernel, grid, 32 * kWarps, 0, stream, p); };
  return p.c.kv_dtype == MLA_KV_BF16            ? launch(mla_cache_weights_kernel<MLA_KV_BF16>)
         : p.c.kv_dtype == MLA_KV_FP8_E4M3_E8M0 ? launch(mla_cache_weights_kernel<MLA_KV_FP8_E4M3_E8M0>)
                                                : launch(mla_cache_weights_kernel<MLA_KV_FP4_E2M1_E8M0>);
}

}  // namespace mla
