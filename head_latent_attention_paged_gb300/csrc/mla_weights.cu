// The weight that queries give to each cached row: a matrix product whose epilogue
// sums exponentials, on pairs of CTAs (tcgen05, cta_group::2).
//
//     S^T [256 tokens x N rows] = K [256 x 576] Q^T, N up to 256
//     w_t += sum over rows r of exp2(scale s_rt - lse_r log2 e)
//
// Tokens are the rows of the accumulator, 128 in each CTA, so that a token's sum
// over queries runs along its own lane: no exchange between lanes, and one thread
// adds a token's weight in a fixed order.  Both operands stream through one ring in
// chunks of 64 of the 576 values.  Work is cut between clusters at tiles of 256
// tokens, each cluster walking all queries of its tiles.
//
// One read of the cache bounds a decode step (64 requests of 4,608 rows, 20 heads: 67 us,
// 5.1 TB/s, 51 us at the copy rate), the products a prompt's end (64 tokens of 20 heads
// behind 32,768: 38 us, 1,260 TFLOP/s, where each pair has 1 or 2 tiles and starts and
// ends idle), the three launches a few drafts over a quantised cache (26 us).  A decode
// step over a quantised cache pays for rows expanded in HBM that it uses once (64 requests
// of 4,608 rows: FP8 152 us, FP4 139), short whole prompts for cuts at tiles alone (2 of
// 1,283 tokens, 32 heads: 12 tiles for 76 pairs, 413 us).
#include <cuda_runtime.h>

#include "mla_chunk_internal.h"
#include "mla_chunk_tiles.cuh"

namespace mla {

namespace {

constexpr int kTokens = 2 * kTileRows;  // of a pair's tile
constexpr int kMaxN = 256;              // rows (token, head) of a block
// The ring: a slot has a chunk of the CTA's tokens and one of its half of a block's
// rows, as many slots as there is room for (a multiple of 3, chunks being loaded three
// at a time): 6 for blocks of 256 rows, 9 where no request has more than 128, as in a
// decode step, which memory bounds (with 6: decode step of 64 75 us).
// Two warps of each CTA fill a slot, and a wait by parity cannot tell a use from the one
// two before it.  Neither warp can be that far ahead: `full` counts the arrivals of both
// (the leader's) and the bytes of all four, so that the MMAs that free a slot wait for
// every one of them, and none passes `empty` for the next use before all have filled this one.
constexpr int kABytes = kTileRows * 128;
constexpr int kMaxSlots = 9, kRingBytes = 216 * 1024;
constexpr int kSumWarps = 8;
constexpr int kThreads = 128 + 32 * kSumWarps;   // 4 warps that load and issue
constexpr int kBoxRows = 32;            // of the queries' boxes

struct WeightsKernelParams {
  WeightsParams w;
  const int2* dense;            // ChunkWorkspace::starts
  int32_t box_rows;             // cached rows of a box: min(page, 128)
};
struct Maps {
  CUtensorMap q, k;
};

// A request's tiles and what each costs: a read of its rows and its products, in
// the latter's time for 64 rows of queries.
struct Tiles {
  ChunkRequest r;
  int32_t end, tiles;           // end: weights that there are
  int64_t cost;
  Tiles() = default;
  __device__ __forceinline__ Tiles(const WeightsKernelParams& p, int32_t b) : r(p.w.c, b) {
    end = static_cast<int32_t>(min(static_cast<int64_t>(r.len), p.w.stride));
    tiles = static_cast<int32_t>((static_cast<int64_t>(end) + kTokens - 1) / kTokens);
    cost = 1 + (r.count > 0 ? 5 + (r.count * p.w.c.heads + 63) / 64 : 0);
  }
};

struct Control {
  uint64_t full[kMaxSlots], empty[kMaxSlots]; // full: in the leader, both CTAs' bytes of both operands
  uint64_t d_full[2], d_free[2];
  float neg_lse[2][kMaxN];              // [block's parity][row]: -lse log2 e, -inf for no row
  int32_t seen[2][kMaxN];
  float sums[2][kTileRows];
  int64_t warp_sum[kThreads / 32];
  int32_t cut[2][2];                    // begin and end: request, tile
  Tiles tiles;                          // of the first request
  int32_t most_rows;                    // (token, head) of a request
  uint32_t tmem;
  int abort;
};
constexpr int kOffControl = kRingBytes, kSmemBytes = kOffControl + sizeof(Control);
static_assert(kSmemBytes <= kMaxSmemBytes, "shared memory");

__device__ __forceinline__ uint8_t* shared_base() {
  extern __shared__ __align__(1024) uint8_t smem[];
  return smem;
}
__device__ __forceinline__ Control* control() { return reinterpret_cast<Control*>(shared_base() + kOffControl); }
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
  return mbar_test(bar, parity) || wait_on(bar, parity, &control()->abort, status);
}

// A tile of a request and the blocks of queries that see any of it.
struct Unit {
  int32_t b, tile, end, limit;
  int32_t row0, rows;           // the request's first row (token, head) of all, and how many
  int32_t block, blocks;        // blocks of 256 rows: from the first that sees the tile
  int32_t len, count;
};
struct Walk {
  int32_t b, tile, of;
  Tiles t;
};
__device__ __noinline__ bool next_unit(const WeightsKernelParams& p, const int32_t* end, Walk* w, Unit* u) {
  const ChunkParams& c = p.w.c;
  while (w->b < end[0] || (w->b == end[0] && w->tile < end[1])) {
    if (w->of != w->b) {
      w->t = Tiles(p, w->b);
      w->of = w->b;
    }
    if (w->tile >= w->t.tiles) {
      ++w->b;
      w->tile = 0;
      continue;
    }
    const ChunkRequest& r = w->t.r;
    const int32_t rows = r.count * c.heads;
    // the first token of the request that sees the tile's first row
    const int64_t first = c.causal ? static_cast<int64_t>(w->tile) * kTokens - (r.len - r.count) : 0;
    const int32_t from = static_cast<int32_t>(min(max(first, int64_t{0}), static_cast<int64_t>(r.count)));
    *u = Unit{w->b, w->tile, w->t.end, rows_there(p.dense, r, w->b), r.first * c.heads, rows,
              from * c.heads / kMaxN, (rows + kMaxN - 1) / kMaxN, r.len, r.count};
    if (from == r.count) u->block = u->blocks;
    ++w->tile;
    return true;
  }
  return false;
}

__device__ __forceinline__ int block_columns(const Unit& u, int32_t block) {   // N of its MMAs
  return min(kMaxN, (u.rows - block * kMaxN + 63) / 64 * 64);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_cache_weights_kernel(const __grid_constant__ WeightsKernelParams p, const __grid_constant__ Maps maps) {
  uint8_t* const smem = shared_base();
  Control* const ctl = control();
  const ChunkParams& c = p.w.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(&ctl->full[i], 2);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->d_full[i], 1);
      mbar_init(&ctl->d_free[i], kSumWarps);   // a group's four of each CTA
    }
    ctl->abort = 0;
    ctl->most_rows = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
  }
  // the pair allocates together: not before both CTAs run
  __syncthreads();
  cluster_sync_all();
  if (warp == 2) pair_tmem_alloc(&ctl->tmem, 512);
  after_predecessor();

  // the cost prefix over requests, and this cluster's cuts: half of the threads for
  // its begin, half for its end, found by the thread in whose requests it lies
  {
    constexpr int kSide = kThreads / 2;
    const int side = threadIdx.x / kSide, i = threadIdx.x % kSide;
    const int32_t batch = c.batch, each = (batch + kSide - 1) / kSide;
    const int32_t lo = min(i * each, batch), hi = min(lo + each, batch);
    int64_t sum = 0;
    int32_t most = 0;
    bool bad = false;
    Tiles t;
    for (int32_t b = hi; b-- > lo;) {     // down, so that t ends as the first one's
      t = Tiles(p, b);
      bad |= t.r.bad || rows_there(p.dense, t.r, b) < t.r.len;
      sum += t.tiles * t.cost;
      most = max(most, t.r.count * c.heads);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (side == 0 && lane == 0 && most > 0) atomicMax(&ctl->most_rows, most);
    if (bad && blockIdx.x == 0 && c.status) atomicOr(c.status, MLA_STATUS_BAD_INDEX);
    int64_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) ctl->warp_sum[warp] = upto;
    if (i == 0) {                         // a cut at the end of the work lies in no request
      ctl->cut[side][0] = batch;
      ctl->cut[side][1] = 0;
    }
    __syncthreads();
    int64_t at = upto - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kSide / 32; ++w) {
      const int64_t of = ctl->warp_sum[side * (kSide / 32) + w];
      if (w < i / 32) at += of;
      total += of;
    }
    // the same for both sides of a cut, and not descending: that is all it has to be
    const int k = cluster + side;
    const float share = static_cast<float>(total) * (static_cast<float>(k) / static_cast<float>(clusters));
    const int64_t x = k == clusters ? total : min(static_cast<int64_t>(share), total);
    if (at <= x && x < at + sum) {
      int32_t b = lo;
      while (x >= at + t.tiles * t.cost) {
        at += t.tiles * t.cost;
        t = Tiles(p, ++b);
      }
      ctl->cut[side][0] = b;
      ctl->cut[side][1] = min(static_cast<int32_t>(static_cast<float>(x - at) / static_cast<float>(t.cost)), t.tiles);
      if (side == 0) ctl->tiles = t;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();           // both CTAs have their half of tensor memory
  tc_fence_after();

  const uint32_t tmem = ctl->tmem;
  uint32_t* const status = c.status;
  const uint32_t slot_bytes = kABytes + min(kMaxN, (ctl->most_rows + 63) / 64 * 64) * 64;
  const uint32_t slots = min(kMaxSlots, static_cast<int>(kRingBytes / slot_bytes / 3 * 3));
  Walk walk;
  walk.b = walk.of = ctl->cut[0][0];
  walk.tile = ctl->cut[0][1];
  walk.t = ctl->tiles;
  const int32_t* const end = ctl->cut[1];
  Unit u;
  bool ok = true;

  if (warp == 0 || warp == 3) {
    // warp 0: this CTA's 128 cached rows, warp 3: its half of the block's queries;
    // three chunks at a time, a lane for each of their boxes (8 of cached rows or 4
    // of queries a chunk at most).  A unit is looked up one ahead.
    const bool cached = warp == 0;
    const uint32_t full_at = mapa_shared(smem_u32(ctl->full), 0);
    const int chunk = lane >> 3, box = lane & 7;
    uint32_t slot = 0, phase = 1;         // phase: of `empty`, at first complete
    Unit next;
    TilePages pages;
    const auto advance = [&]() {          // the next unit with blocks, and its pages
      while (next_unit(p, end, &walk, &next)) {
        if (next.block >= next.blocks) continue;
        pages.load(c, next.b, next.limit, 2 * next.tile + static_cast<int32_t>(rank), lane);
        return true;
      }
      return false;
    };
    bool more = advance();
    while (ok && more) {
      u = next;
      const int32_t tile = 2 * u.tile + static_cast<int32_t>(rank);
      const TileRows rows(c, u.limit, tile, pages, -1, lane);
      if (cached && pages.bad(c) && lane == 0 && status) atomicOr(status, MLA_STATUS_BAD_PAGE);
      more = advance();
      // Slots that hold no row of the request are read all the same, pages that are not
      // there from the pool's start: a token's sums see no other token's row.
      int32_t boxed = max(__shfl_sync(0xffffffffu, rows.base, (box * (p.box_rows >> 4)) & 7), 0);
      if (p.dense) boxed = rows.left > 0 ? p.dense[u.b].x + tile * kTileRows : 0;
#pragma unroll 1
      for (int32_t block = u.block; ok && block < u.blocks; ++block) {
        const int32_t half = block_columns(u, block) / 2;
        const int32_t row = u.row0 + block * kMaxN + half * static_cast<int32_t>(rank) + kBoxRows * box;
        const int boxes = cached ? kTileRows / p.box_rows : half / kBoxRows;
        const uint32_t bytes = cached ? kABytes : half * 128;
#pragma unroll 1
        for (int k = 0; ok && k < kChunks; k += 3) {
          const uint32_t mine = slot + chunk;   // this lane's
          bool todo = chunk < 3 && box < boxes;
          for (uint32_t n = 1; __any_sync(0xffffffffu, todo); ++n) {
            if (todo && mbar_poll(&ctl->empty[mine], phase)) {
              if (box == 0 && rank == 0) mbar_arrive_expect_tx(&ctl->full[mine], 2 * bytes);
              uint8_t* const dst = smem + mine * slot_bytes;
              if (cached)
                pair_tma_load_3d(dst + box * p.box_rows * 128, &maps.k, full_at + 8 * mine, 0, boxed, k + chunk);
              else
                pair_tma_load_3d(dst + kABytes + box * (kBoxRows * 128), &maps.q, full_at + 8 * mine, 0, row, k + chunk);
              todo = false;
            }
            if ((n & 1023u) == 0) {     // the slowest of them, with a limit
              bool there = true;
              if (todo) there = wait_on(&ctl->empty[mine], phase, &ctl->abort, status);
              ok = __all_sync(0xffffffffu, there);
              if (!ok) break;
            }
          }
          slot += 3;
          if (slot == slots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const MatrixWords a0(smem, 16, 1024);
      uint32_t slot = 0, phase = 0, done = 0;
      while (ok && next_unit(p, end, &walk, &u)) {
#pragma unroll 1
        for (int32_t block = u.block; ok && block < u.blocks; ++block, ++done) {
          const uint32_t idesc = make_idesc_bf16(kTokens, block_columns(u, block), false, false);
          const uint32_t col = tmem + kMaxN * (done & 1);
          ok = done < 2 || __all_sync(0xffffffffu, wait(&ctl->d_free[done & 1], ((done >> 1) - 1) & 1, status));
#pragma unroll 1
          for (int k = 0; ok && k < kChunks; ++k) {
            ok = __all_sync(0xffffffffu, wait(&ctl->full[slot], phase, status));
            tc_fence_after();
            const uint32_t a = a0.lo + ((slot * slot_bytes) >> 4), b = a + (kABytes >> 4);
#pragma unroll
            for (int m = 0; m < 4; ++m) pair_mma_bf16(col, a + 2 * m, a0.hi, b + 2 * m, a0.hi, idesc, k > 0 || m > 0);
            pair_commit(&ctl->empty[slot]);
            if (++slot == slots) {
              slot = 0;
              phase ^= 1;
            }
          }
          pair_commit(&ctl->d_full[done & 1]);
        }
      }
    }
  } else if (warp >= 4) {
    // Sums: a lane of tensor memory is a token.  Blocks go to the warps 4 .. 7 and 8 ..
    // 11 in turn, each with an accumulator of its own: what stands between a group's
    // blocks (a unit's end, the next one's look-up) runs beside the other's sums.
    const int quad = warp & 3, l = quad * 32 + lane, group = (warp >> 2) - 1;
    const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + kMaxN * group;
    const uint32_t free_bar = mapa_shared(smem_u32(&ctl->d_free[group]), 0);
    const float2 scale2 = make_float2(c.scale_log2, c.scale_log2);
    float* const neg = ctl->neg_lse[group];
    int32_t* const seen = ctl->seen[group];
    uint32_t done = 0, joined = 0;
    bool failed = false;
    while (next_unit(p, end, &walk, &u)) {
      const int32_t blocks = u.blocks - u.block;
      // a unit of one block is its group's alone
      if (blocks < 2 && (blocks == 0 ? 0 : static_cast<int>(done & 1)) != group) {
        done += blocks;
        continue;
      }
      const int64_t first = static_cast<int64_t>(u.tile) * kTokens + kTileRows * rank, t = first + l;
      const ChunkRequest r(u.len, u.count);
      const bool writes = blocks < 2 || group == 0;
      // used at the end: what it is added to, and whether the row is there
      const int64_t out = u.b * p.w.stride + t;
      const float before = writes && t < u.end && p.w.in ? p.w.in[out] : 0.f;
      const int32_t page = writes && t < min(u.end, u.limit)
                               ? c.block_table[static_cast<int64_t>(u.b) * c.max_pages + (t >> c.page_shift)] : -1;
      float2 acc[2] = {};
#pragma unroll 1
      for (int32_t block = u.block; block < u.blocks; ++block, ++done) {
        if (static_cast<int>(done & 1) != group) continue;
        const int columns = block_columns(u, block);
#pragma unroll 1
        for (int e = l; e < columns; e += kTileRows) {
          const int32_t row = block * kMaxN + e;
          const float lse = row < u.rows ? p.w.lse[u.row0 + row] : INFINITY;
          neg[e] = lse == -INFINITY ? -INFINITY : lse * -1.4426950408889634f;   // no weight from a row that saw nothing
          seen[e] = row < u.rows ? r.seen(row / c.heads, c.causal) : 0;
        }
        failed |= !wait(&ctl->d_full[group], (done >> 1) & 1, status);
        failed = named_bar_or(1 + group, 128, failed);   // agreed on by the group
        if (failed) break;
        tc_fence_after();
        const bool all = seen[0] >= first + kTileRows && (block + 1) * kMaxN <= u.rows;
#pragma unroll 1
        for (int k = 0; k < columns; k += 32) {
          uint32_t x[32];
          tmem_ld32(from + k, x);
          const float4* n4 = reinterpret_cast<const float4*>(neg + k);
          float v[32];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 n = n4[q];
            const float2 a = __ffma2_rn(make_float2(__uint_as_float(x[4 * q]), __uint_as_float(x[4 * q + 1])), scale2, make_float2(n.x, n.y));
            const float2 b = __ffma2_rn(make_float2(__uint_as_float(x[4 * q + 2]), __uint_as_float(x[4 * q + 3])), scale2, make_float2(n.z, n.w));
            v[4 * q] = exp2_approx(a.x);
            v[4 * q + 1] = exp2_approx(a.y);
            v[4 * q + 2] = exp2_approx(b.x);
            v[4 * q + 3] = exp2_approx(b.y);
          }
          if (!all) {                     // rows that do not see the token, and none
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] = t < seen[k + q] ? v[q] : 0.f;
          }
#pragma unroll
          for (int q = 0; q < 16; ++q) acc[q & 1] = __fadd2_rn(acc[q & 1], make_float2(v[2 * q], v[2 * q + 1]));
        }
        tc_fence_before();
        named_bar_or(1 + group, 128, false);   // neg and seen have been read
        if (lane == 0) cluster_mbar_arrive(free_bar);
      }
      float sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
      if (blocks >= 2) {                  // both groups have a part
        float* const other = ctl->sums[joined++ & 1];
        if (group == 1) other[l] = sum;
        if (named_bar_or(3, 32 * kSumWarps, failed)) break;
        sum += group == 0 ? other[l] : 0.f;
      } else if (failed) {
        continue;               // to where the other group waits, or the end
      }
      if (writes && t < u.end) p.w.out[out] = before + (page >= 0 && page < c.num_pages ? sum : 0.f);
    }
  }
  __syncwarp();
  volatile int* const abort = &ctl->abort;
  if (*abort) let_copies_land();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();           // neither CTA leaves while the other may still write to it
  tc_fence_after();
  if (warp == 2) pair_tmem_dealloc(tmem, 512);
  __syncthreads();
  cluster_sync_all();           // nor leave before both have given it back
}

}  // namespace

cudaError_t launch_cache_weights(const WeightsParams& w, const ChunkWorkspace& ws, cudaStream_t stream) {
  WeightsKernelParams p;
  p.w = w;
  p.dense = ws.starts;
  p.box_rows = ws.starts ? kTileRows : 1 << w.c.page_shift;
  const void* rows = ws.starts ? static_cast<const void*>(ws.rows) : w.c.kv;
  const uint64_t count = ws.starts ? static_cast<uint64_t>(ws.capacity > 0 ? ws.capacity : 1)
                                   : static_cast<uint64_t>(w.c.num_pages) << w.c.page_shift;
  const uint64_t queries = static_cast<uint64_t>(w.c.tokens > 0 ? w.c.tokens : 1) * w.c.heads;
  Maps maps;
  if (!make_map_chunks_bf16(&maps.q, w.c.q, kDqk, queries, kDqk * 2, kBoxRows, 1) ||
      !make_map_chunks_bf16(&maps.k, rows, kDqk, count, kDqk * 2, p.box_rows, 1))
    return cudaErrorInvalidValue;
  cudaError_t err = set_smem_attr_once(reinterpret_cast<const void*>(mla_cache_weights_kernel), kSmemAttrWeights, kSmemBytes);
  if (err != cudaSuccess) return err;
  return launch_dependent(mla_cache_weights_kernel, dim3(2 * ws.clusters), kThreads, kSmemBytes, stream, p, maps);
}

}  // namespace mla
