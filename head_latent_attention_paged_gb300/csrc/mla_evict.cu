// Eviction: each request's slots selected by weight, and the kept rows behind
// the budget moved into the slots below it that became free.
#include <cuda_runtime.h>

#include "mla_chunk_internal.h"

namespace mla {

namespace {

constexpr int kSelectThreads = 1024;
constexpr int kMoveWarps = 4;

// A slot's rank as an unsigned number: protected slots above every weight,
// NaN below, -0 as 0.
__device__ __forceinline__ uint32_t rank_key(float w, bool safe) {
  if (safe) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const uint32_t bits = __float_as_uint(w + 0.f);
  return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
}

// Exclusive prefix of v over the block's threads, and the block's total.
__device__ __forceinline__ int block_prefix(int v, int* total) {
  __shared__ int sums[kSelectThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < kSelectThreads / 32; ++i) {
    if (i < warp) before += sums[i];
    all += sums[i];
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

__global__ void __launch_bounds__(kSelectThreads) mla_evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int hist[256], s_newest, s_digit, s_left;
  after_predecessor();
  const int b = blockIdx.x, tid = threadIdx.x;
  const float* w = p.weights + b * p.stride;
  const int32_t* pos = p.positions + b * p.stride;
  float* w_out = p.weights_out + b * p.stride;
  int32_t* pos_out = p.positions_out + b * p.stride;
  const int64_t most = min(static_cast<int64_t>(p.max_pages) << p.page_shift, p.stride);
  const int32_t given = p.lens[b];
  const int32_t n = static_cast<int32_t>(min(max(static_cast<int64_t>(given), int64_t{0}), most));
  if (n != given && p.status && tid == 0) atomicOr(p.status, MLA_STATUS_BAD_INDEX);
  const int32_t budget = min(n, p.budget);
  int32_t* moves = p.moves + b * p.most_moves * 2;
  int count = 0;
  if (n > budget) {
    if (tid == 0) s_newest = -1;
    __syncthreads();
    int newest = -1;
    for (int t = tid; t < n; t += kSelectThreads) newest = max(newest, pos[t]);
    atomicMax(&s_newest, newest);
    __syncthreads();
    const int64_t border = static_cast<int64_t>(s_newest) - p.recent;
    const auto key_of = [&](int t) { return rank_key(w[t], pos[t] < p.sinks || pos[t] > border); };
    // the budget-th greatest key, eight bits at a time
    uint32_t prefix = 0, mask = 0;
    int left = budget;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int t = tid; t < n; t += kSelectThreads) {
        const uint32_t k = key_of(t);
        if ((k & mask) == prefix) atomicAdd(&hist[k >> shift & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255;
        while (hist[d] < left) left -= hist[d--];
        s_digit = d;
        s_left = left;
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(s_digit) << shift;
      mask |= 255u << shift;
      left = s_left;
      __syncthreads();
    }
    // in the order of slots: the first `left` of those that equal it are kept;
    // the i-th free slot below the budget takes the i-th kept row behind it
    int equal = 0, holes = 0, movers = 0;
    for (int base = 0; base < n; base += kSelectThreads) {
      const int t = base + tid;
      const uint32_t k = t < n ? key_of(t) : 0;
      int total;
      const bool tie = t < n && k == prefix;
      const int rank = equal + block_prefix(tie, &total);
      equal += total;
      const bool kept = t < n && (k > prefix || (tie && rank < left));
      const bool hole = t < budget && !kept, mover = kept && t >= budget;
      const int h = holes + block_prefix(hole, &total);
      holes += total;
      if (hole) moves[2 * h] = t;
      const int m = movers + block_prefix(mover, &total);
      movers += total;
      if (mover) moves[2 * m + 1] = t;
    }
    count = holes;
    __syncthreads();
    for (int i = tid; i < count; i += kSelectThreads) {
      const int to = moves[2 * i], from = moves[2 * i + 1];
      w_out[to] = w[from];
      pos_out[to] = pos[from];
    }
    __syncthreads();
  }
  // what stays, where the outputs are other arrays, and the slots given up
  if (w_out != w || pos_out != pos) {
    int next = 0;   // holes below t
    for (int t = tid; t < budget; t += kSelectThreads) {
      while (next < count && moves[2 * next] < t) ++next;
      if (next < count && moves[2 * next] == t) continue;
      w_out[t] = w[t];
      pos_out[t] = pos[t];
    }
  }
  for (int t = budget + tid; t < n; t += kSelectThreads) {
    w_out[t] = 0.f;
    pos_out[t] = -1;
  }
  if (tid == 0) {
    p.counts[b] = count;
    p.lens_out[b] = budget;
  }
}

// One warp per row: its bytes in units of 2, which divide every format's rows.
__global__ void __launch_bounds__(32 * kMoveWarps) mla_evict_move_kernel(const __grid_constant__ EvictParams p) {
  const int lane = threadIdx.x & 31;
  after_predecessor();
  const int b = blockIdx.y, count = p.counts[b];
  const int32_t* moves = p.moves + b * p.most_moves * 2;
  const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_pages;
  for (int i = blockIdx.x * kMoveWarps + (threadIdx.x >> 5); i < count; i += gridDim.x * kMoveWarps) {
    const int to = moves[2 * i], from = moves[2 * i + 1];
    const int32_t pt = table[to >> p.page_shift], pf = table[from >> p.page_shift];
    if (pt < 0 || pt >= p.num_pages || pf < 0 || pf >= p.num_pages) {
      if (p.status && lane == 0) atomicOr(p.status, MLA_STATUS_BAD_PAGE);
      continue;
    }
    const int in_page = (1 << p.page_shift) - 1;
    const uint16_t* src = reinterpret_cast<const uint16_t*>(
        p.kv + ((static_cast<int64_t>(pf) << p.page_shift) + (from & in_page)) * p.row_bytes);
    uint16_t* dst = reinterpret_cast<uint16_t*>(
        p.kv + ((static_cast<int64_t>(pt) << p.page_shift) + (to & in_page)) * p.row_bytes);
    for (int k = lane; k < p.row_bytes / 2; k += 32) dst[k] = src[k];
  }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictParams& p, cudaStream_t stream) {
  cudaError_t err = launch_dependent(mla_evict_select_kernel, dim3(p.batch), kSelectThreads, 0, stream, p);
  if (err != cudaSuccess) return err;
  return launch_dependent(mla_evict_move_kernel, dim3(128, p.batch), 32 * kMoveWarps, 0, stream, p);
}

}  // namespace mla
