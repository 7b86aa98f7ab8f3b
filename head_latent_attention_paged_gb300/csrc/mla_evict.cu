// Eviction: each request's slots selected by weight, and the kept rows behind the
// budget moved into the slots below it that became free.
//
// The budget-th greatest weight is found digit by digit (11, 11 and 10 bits of an
// order-preserving integer) from counts; its equals are taken in the order of slots.
// A cluster of CTAs holds a request: every slot's key is made once and stays in
// shared memory, counts and prefixes go through the cluster's shared memory.  Only
// rows that leave a slot behind the budget move, so a cache that has grown by a few
// rows over its budget moves a few rows.
#include <cuda_runtime.h>

#include "mla_chunk_internal.h"
#include "sm103_ptx.cuh"

namespace mla {

namespace {

constexpr int kThreadsShift = 10, kThreads = 1 << kThreadsShift, kWarps = kThreads / 32;
constexpr int kBins = 2048, kCoarse = kBins / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxKeys = 49152;         // of a CTA, in shared memory; those behind are made again
constexpr int kMoveWarps = 4;

// A slot's rank as an unsigned number: protected slots above every weight, NaN
// below, -0 as 0.
__device__ __forceinline__ uint32_t rank_key(float w, bool safe) {
  if (safe) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const uint32_t bits = __float_as_uint(w + 0.f);
  return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
}

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ int64_t ld_cluster_two(uint32_t addr) {
  int64_t v;
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

struct Shared {
  int hist[3][kBins];           // of each digit
  alignas(8) int coarse[3][kCoarse];      // of 32 bins each
  int newest, digit, left, ties;
  int tie[kWarps], hole[kWarps], mover[kWarps];   // of each warp
  int all[3];                   // of this CTA
};

// The sum of v over the lanes behind this one.
__device__ __forceinline__ int behind(int v) {
  const int lane = threadIdx.x & 31, own = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_down_sync(0xffffffffu, v, o);
    if (lane + o < 32) v += y;
  }
  return v - own;
}

// The bin that holds the left-th greatest key, from the cluster's counts: the 32 bins
// around it first, then it, 64 and 32 counts of each CTA (all 2,048 of eight CTAs took
// 2 us a digit).  One warp; the loads of all CTAs are on their way at once.
__device__ __noinline__ void find_digit(Shared* s, int digit, int clusters, int left) {
  const int lane = threadIdx.x & 31;
  int64_t two[kMaxCluster], both = 0;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    two[r] = r < clusters ? ld_cluster_two(mapa_shared(smem_u32(&s->coarse[digit][2 * lane]), r)) : 0;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) both += two[r];   // neither half carries: below 2^31
  const int lo = static_cast<int>(both), hi = static_cast<int>(both >> 32);
  int before = behind(lo + hi);
  const bool second = left > before + hi;
  const uint32_t here = __ballot_sync(0xffffffffu, before < left && left <= before + lo + hi);
  const int at = __ffs(here) - 1;
  const int coarse = __shfl_sync(0xffffffffu, 2 * lane + !second, at);
  left -= __shfl_sync(0xffffffffu, before + (second ? hi : 0), at);
  int count[kMaxCluster], sum = 0;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    count[r] = r < clusters ? ld_cluster(mapa_shared(smem_u32(&s->hist[digit][32 * coarse + lane]), r)) : 0;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) sum += count[r];
  before = behind(sum);
  if (before < left && left <= before + sum) {
    s->digit = 32 * coarse + lane;
    s->left = left - before;
    s->ties = sum;
  }
}

// What stands before this warp: counts[w] of the warps before it in the CTA, and the
// CTAs' `all` before it in the cluster.  Warp-wide; after a cluster barrier.
__device__ __forceinline__ int before_warp(const int* counts, const int* all, uint32_t rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = lane < warp ? counts[lane] : 0;
  if (lane < static_cast<int>(rank)) v += ld_cluster(mapa_shared(smem_u32(all), lane));
  return __reduce_add_sync(0xffffffffu, v);
}

// One cluster per request (kMaxKeys slots a CTA without making keys again; 32,768
// slots cut to 4,096 by eight CTAs and moved 19 us, by one CTA that read them again
// for every digit 410 us).  Bound by latency: 13 us are six barriers of the cluster and
// what lies between them (a digit 1.5 us), not the 0.3 MB read.
__global__ void __launch_bounds__(kThreads, 1) mla_evict_select_kernel(const __grid_constant__ EvictParams p, const int cluster_shift, const int cap) {
  extern __shared__ uint32_t keys[];
  __shared__ Shared s;
  after_predecessor();
  const int clusters = 1 << cluster_shift, b = blockIdx.x >> cluster_shift;   // CTAs of a request
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = blockIdx.x & (clusters - 1);
  const float* w = p.weights + b * p.stride;
  const int32_t* pos = p.positions + b * p.stride;
  float* w_out = p.weights_out + b * p.stride;
  int32_t* pos_out = p.positions_out + b * p.stride;
  const int64_t most = min(static_cast<int64_t>(p.max_pages) << p.page_shift, p.stride);
  const int32_t given = p.lens[b];
  const int32_t n = static_cast<int32_t>(min(max(static_cast<int64_t>(given), int64_t{0}), most));
  const int32_t budget = min(n, p.budget);
  // each warp has consecutive slots, 32 at a time
  const int32_t each = static_cast<int32_t>((static_cast<int64_t>(n) + clusters * kThreads - 1) >> (cluster_shift + kThreadsShift)) * 32;
  const int64_t at = (static_cast<int64_t>(rank) * kWarps + warp) * each;
  const int32_t first = static_cast<int32_t>(min(at, static_cast<int64_t>(n)));
  const int32_t steps = (min(each, n - first) + 31) / 32;
  int32_t* moves = p.moves + b * p.most_moves * 2;
  if (rank == 0 && tid == 0 && n != given && p.status) atomicOr(p.status, MLA_STATUS_BAD_INDEX);

  int32_t moved = 0;
  if (n > budget) {             // the same for the whole cluster
    if (tid == 0) s.newest = -1;
    for (int i = tid; i < 3 * kBins; i += kThreads) (&s.hist[0][0])[i] = 0;
    if (tid < 3 * kCoarse) (&s.coarse[0][0])[tid] = 0;
    __syncthreads();
    const int own = warp * each;          // of this CTA's keys
    int newest = -1;
#pragma unroll 4
    for (int k = 0; k < steps; ++k) {
      const int t = first + 32 * k + lane, i = own + 32 * k + lane;
      if (t >= n) continue;
      const int position = pos[t];
      const float weight = w[t];
      newest = max(newest, position);
      if (i < cap) keys[i] = __float_as_uint(weight);
      if (t < budget) {         // for rows that stay; the others' slots are written again
        w_out[t] = weight;
        pos_out[t] = position;
      }
    }
    newest = __reduce_max_sync(0xffffffffu, newest);
    if (lane == 0) atomicMax(&s.newest, newest);
    cluster_sync_all();
    newest = lane < clusters ? ld_cluster(mapa_shared(smem_u32(&s.newest), lane)) : -1;
    newest = __reduce_max_sync(0xffffffffu, newest);
    const int64_t border = static_cast<int64_t>(newest) - p.recent;
    const auto make_key = [&](int t, float weight) { return rank_key(weight, pos[t] < p.sinks || pos[t] > border); };
    const auto key_at = [&](int k) {
      const int i = own + 32 * k + lane;
      return i < cap ? keys[i] : make_key(first + 32 * k + lane, w[first + 32 * k + lane]);
    };
    // the budget-th greatest key
    uint32_t found = 0, mask = 0;
    int left = budget, ties = 0;
    for (int digit = 0; digit < 3; ++digit) {
      const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bits = digit == 2 ? 10 : 11;
      for (int k = 0; k < steps; ++k) {
        const int t = first + 32 * k + lane;
        if (t >= n) continue;
        uint32_t key;
        if (digit == 0) {
          const int i = own + 32 * k + lane;
          key = make_key(t, i < cap ? __uint_as_float(keys[i]) : w[t]);
          if (i < cap) keys[i] = key;
        } else {
          key = key_at(k);
        }
        if ((key & mask) == found) {
          const int bin = key >> shift & ((1 << bits) - 1);
          atomicAdd(&s.hist[digit][bin], 1);
          atomicAdd(&s.coarse[digit][bin >> 5], 1);
        }
      }
      cluster_sync_all();
      if (warp == 0) find_digit(&s, digit, clusters, left);
      __syncthreads();
      found |= static_cast<uint32_t>(s.digit) << shift;
      mask |= ((1u << bits) - 1u) << shift;
      left = s.left;
      ties = s.ties;
    }
    // equal ones: the first `left` of `ties` in the order of slots
    int ties_before = 0;
    if (ties != left) {
      int count = 0;
      for (int k = 0; k < steps; ++k) {
        const int t = first + 32 * k + lane;
        count += __popc(__ballot_sync(0xffffffffu, t < n && key_at(min(k, steps - 1)) == found));
      }
      if (lane == 0) s.tie[warp] = count;
      __syncthreads();
      if (warp == 0) {
        const int all = __reduce_add_sync(0xffffffffu, s.tie[lane]);
        if (lane == 0) s.all[0] = all;
      }
      cluster_sync_all();
      ties_before = before_warp(s.tie, &s.all[0], rank);
    }
    const auto kept_at = [&](int k, int* tied) {   // tied: of this warp so far
      const int t = first + 32 * k + lane;
      const uint32_t key = t < n ? key_at(k) : 0u;
      const bool tie = t < n && key == found;
      const uint32_t same = __ballot_sync(0xffffffffu, tie);
      const int at_tie = ties_before + *tied + __popc(same & ((1u << lane) - 1u));
      *tied += __popc(same);
      return t < n && (key > found || (tie && (ties == left || at_tie < left)));
    };
    // the i-th free slot below the budget takes the i-th kept row behind it
    int holes = 0, movers = 0, tied = 0;
    for (int k = 0; k < steps; ++k) {
      const int t = first + 32 * k + lane;
      const bool kept = kept_at(k, &tied);
      holes += __popc(__ballot_sync(0xffffffffu, t < budget && !kept));
      movers += __popc(__ballot_sync(0xffffffffu, t >= budget && kept));
    }
    if (lane == 0) {
      s.hole[warp] = holes;
      s.mover[warp] = movers;
    }
    __syncthreads();
    if (warp == 0) {
      const int h = __reduce_add_sync(0xffffffffu, s.hole[lane]), m = __reduce_add_sync(0xffffffffu, s.mover[lane]);
      if (lane == 0) {
        s.all[1] = h;
        s.all[2] = m;
      }
    }
    cluster_sync_all();
    const int first_hole = before_warp(s.hole, &s.all[1], rank), first_mover = before_warp(s.mover, &s.all[2], rank);
    moved = lane < clusters ? ld_cluster(mapa_shared(smem_u32(&s.all[1]), lane)) : 0;
    moved = __reduce_add_sync(0xffffffffu, moved);
    cluster_arrive();           // what this CTA reads of the others it has read
    holes = first_hole;
    movers = first_mover;
    tied = 0;
    for (int k = 0; k < steps; ++k) {
      const int t = first + 32 * k + lane;
      const bool kept = kept_at(k, &tied), hole = t < budget && !kept, mover = t >= budget && kept;
      const uint32_t h = __ballot_sync(0xffffffffu, hole), m = __ballot_sync(0xffffffffu, mover), below = (1u << lane) - 1u;
      if (hole) moves[2 * (holes + __popc(h & below))] = t;
      if (mover) moves[2 * (movers + __popc(m & below)) + 1] = t;
      holes += __popc(h);
      movers += __popc(m);
      if (t >= budget && t < n && !kept) {   // given up; a mover's slot is cleared as it moves
        w_out[t] = 0.f;
        pos_out[t] = -1;
      }
    }
    cluster_wait();
  } else if (w_out != w || pos_out != pos) {
    for (int k = 0; k < steps; ++k) {
      const int t = first + 32 * k + lane;
      if (t < n) {
        w_out[t] = w[t];
        pos_out[t] = pos[t];
      }
    }
  }
  if (rank == 0 && tid == 0) {
    p.counts[b] = moved;
    p.lens_out[b] = budget;
  }
}

// One warp per row, in units that divide the format's rows; its weight and position
// move with it.  No slot is in two moves.
template <typename Unit, int kRowBytes>
__global__ void __launch_bounds__(32 * kMoveWarps) mla_evict_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kUnits = kRowBytes / sizeof(Unit), kEach = (kUnits + 31) / 32;
  const int lane = threadIdx.x & 31;
  after_predecessor();
  const int b = blockIdx.y, count = p.counts[b];
  const int32_t* moves = p.moves + b * p.most_moves * 2;
  const float* w = p.weights + b * p.stride;
  const int32_t* pos = p.positions + b * p.stride;
  float* w_out = p.weights_out + b * p.stride;
  int32_t* pos_out = p.positions_out + b * p.stride;
  const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_pages;
  const int in_page = (1 << p.page_shift) - 1;
  for (int i = blockIdx.x * kMoveWarps + (threadIdx.x >> 5); i < count; i += gridDim.x * kMoveWarps) {
    const int2 move = reinterpret_cast<const int2*>(moves)[i];
    if (lane == 0) {
      const float weight = w[move.y];
      const int32_t position = pos[move.y];
      w_out[move.x] = weight;
      pos_out[move.x] = position;
      w_out[move.y] = 0.f;
      pos_out[move.y] = -1;
    }
    const int32_t pt = table[move.x >> p.page_shift], pf = table[move.y >> p.page_shift];
    if (pt < 0 || pt >= p.num_pages || pf < 0 || pf >= p.num_pages) {
      if (p.status && lane == 0) atomicOr(p.status, MLA_STATUS_BAD_PAGE);
      continue;
    }
    const Unit* src = reinterpret_cast<const Unit*>(
        p.kv + ((static_cast<int64_t>(pf) << p.page_shift) + (move.y & in_page)) * kRowBytes);
    Unit* dst = reinterpret_cast<Unit*>(
        p.kv + ((static_cast<int64_t>(pt) << p.page_shift) + (move.x & in_page)) * kRowBytes);
    Unit v[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (32 * k + lane < kUnits) v[k] = src[32 * k + lane];
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (32 * k + lane < kUnits) dst[32 * k + lane] = v[k];
  }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictParams& p, cudaStream_t stream) {
  const int64_t slots = p.stride < (static_cast<int64_t>(p.max_pages) << p.page_shift)
                            ? p.stride : static_cast<int64_t>(p.max_pages) << p.page_shift;
  // CTAs for a request: more while there are multiprocessors for them and slots for
  // their threads
  int shift = 0;
  while (1 << shift < kMaxCluster && (int64_t{2} << shift) * p.batch <= kSms && slots > kThreads << shift) ++shift;
  const int cluster = 1 << shift;
  const int64_t own = (slots + cluster * kThreads - 1) / (cluster * kThreads) * kThreads;
  const int cap = static_cast<int>(own < kMaxKeys ? own : kMaxKeys);
  cudaError_t err = set_smem_attr_once(reinterpret_cast<const void*>(mla_evict_select_kernel), kSmemAttrEvict, kMaxKeys * 4);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.batch * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = cap * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, mla_evict_select_kernel, p, shift, cap);
  if (err != cudaSuccess || p.most_moves == 0) return err;
  // rows of all requests over a few blocks a multiprocessor, at most one warp a move
  int64_t blocks = (p.most_moves + kMoveWarps - 1) / kMoveWarps;
  const int64_t fill = (kSms * 8 + p.batch - 1) / p.batch;
  if (blocks > fill) blocks = fill;
  const dim3 grid(static_cast<unsigned>(blocks), p.batch);
  const auto launch = [&](auto kernel) { return launch_dependent(kernel, grid, 32 * kMoveWarps, 0, stream, p); };
  return p.row_bytes == kDqk * 2       ? launch(mla_evict_move_kernel<uint4, kDqk * 2>)
         : p.row_bytes == kFp8RowBytes ? launch(mla_evict_move_kernel<uint16_t, kFp8RowBytes>)
                                       : launch(mla_evict_move_kernel<uint32_t, kFp4RowBytes>);
}

}  // namespace mla
