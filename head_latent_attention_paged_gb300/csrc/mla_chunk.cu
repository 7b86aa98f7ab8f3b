// Attention of a chunk of new tokens over the paged latent cache: pairs of CTAs
// (tcgen05, cta_group::2) over the rows (token, head) of a request.
//
//     s = scale q . row        S [128 x 128] = Q [128 x 576] K^T
//     p = exp2(s - ref)        O [128 x 512] += P [128 x 128] V
//
// over tiles of 128 cached rows, K the whole rows and V their first 512 values.
// The running reference of the exponent moves only when a row's maximum outgrows
// it by 2^8.  P is rounded to bf16: a product's operands have one type, and V, the
// cached rows, is bf16.  O is divided by the sum of the rounded weights, so that
// what is common to a row's roundings cancels; the rest is 0.5e-3 of o (16,384 rows
// seen) to 1.4e-3 (some hundred), where o's own rounding is 1.7e-3.
//
// Why pairs: O takes 128 x 512 accumulators, all of one SM's tensor memory.
// Two CTAs with 64 of the 128 rows each keep O (256 columns: with M = 128 over
// a pair, lanes 64..127 hold the second half of a row's columns) beside two S
// (64 columns each), and the operand that both need is read from both shared
// memories: each CTA loads half of a tile's tokens for S and half of its latent
// columns for O: 278 KB of copies, from L2, for a tile of 147 KB.
//
// Work is a row tile's tiles one after another, and all of it in a line that is cut
// evenly between the pairs; row tiles that were cut are merged by a second kernel.
// Long chunks are bound by the tensor cores (2,048 tokens of 20 heads behind 14,336:
// 710-765 us by machine, 1,790-1,930 TFLOP/s of a library product's 1,905; called again
// and again 823-841 us, at the power limit).  Between two row
// tiles the softmax warps stand for about 3.5 us: the last product, the output's 64 KB,
// the next row tile's first scores.  Chunks with few tiles a row tile pay that often
// (two whole prompts of 1,283 tokens, 5 tiles each: 110 us, 1,040 TFLOP/s).  A single
// short chunk is latency (5 tokens behind 700: 18 us, 7 of them before the first scores).
#include <cuda_runtime.h>

#include "mla_chunk_internal.h"
#include "mla_chunk_tiles.cuh"
#include "mla_rows.cuh"

namespace mla {

namespace {

constexpr int kRows = 128;              // rows of a row tile, 64 in each CTA
constexpr int kHalf = 64;
constexpr int kTok = kTileRows;
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = 128 + 32 * kSoftmaxWarps;   // 4 warps that load and issue
// Two rings, each a tile deep and filled by a warp of its own (a wait by parity
// cannot tell a slot's use from the one two before, so every slot has one warp
// that fills it): K in three 64-wide chunks of this CTA's 64 tokens, V in 32
// tokens of its 256 columns.  A slot holds the same part of every tile.
constexpr int kKChunks = 3, kKSlots = 3, kKSlotBytes = kKChunks * kChunkBytes;
constexpr int kVTokens = 32, kVSlots = 4, kVSlotBytes = kVTokens * 512;
constexpr int kQBytes = kChunks * kChunkBytes;
constexpr int kPBytes = 2 * kChunkBytes;
constexpr int kColO = 0, kColS = 256;   // tensor memory columns
// What a row tile costs besides its tiles, in tokens of one (its queries' load,
// its output): the work is cut where the sum of tokens and this is even.  (256, 384,
// 512, 640: two whole prompts 146, 131, 130, 132 us; 512 tokens behind 8,192 119.5,
// 119.5, 118, 118.4 us; 24 requests over FP8 238, 237, 238, 241 us.)
constexpr int kRowTileCost = 512;
constexpr int kSegments = 4;

struct AttendKernelParams {
  AttendParams a;
  float* part_o;                // [2 * clusters][64][128][8]: eight columns of all rows side by side
  float* part_lse;              // [2 * clusters][128]
  int4* segments;               // [2 * clusters]: kind, first row, rows, 0
  const int2* dense;            // ChunkWorkspace::starts
  int32_t box_rows;             // rows of a K box, min(page, 64)
  int32_t map_rows;             // rows that there are to read
};

// What a cluster's segment slots say to the merge.
enum SegmentKind : int32_t { kNone = 0, kOpens = 1, kContinues = 2, kIdle = 3 };

// A request as the work is cut: its rows, row tiles and what each of them sees.
// (Rows of all requests together are below 2^31 - 128: checked by the host.)
struct Rows {
  ChunkRequest r;
  int32_t limit;                // rows from here on are masked out (expanded rows there are)
  int32_t rows;                 // (token, head)
  int32_t row_tiles;
  Rows() = default;
  __device__ __forceinline__ Rows(const AttendKernelParams& p, int32_t b) : r(p.a.c, b) {
    rows = r.count * p.a.c.heads;
    row_tiles = (rows + kRows - 1) / kRows;
    limit = rows_there(p.dense, r, b);
  }
  __device__ __forceinline__ int32_t tiles(const AttendKernelParams& p, int32_t i) const {
    const int32_t last = min((i + 1) * kRows, rows) - 1;
    const int32_t n = min(r.seen(last / p.a.c.heads, p.a.c.causal), limit);
    return static_cast<int32_t>((static_cast<uint32_t>(n) + kTok - 1) / kTok);
  }
  // heads times the cost of the first i row tiles: what they see, to within a
  // tile each (i below 2^24, heads at most 128: the sum over requests stays
  // below 2^63)
  __device__ __forceinline__ int64_t cost(const AttendKernelParams& p, int64_t i) const {
    const int64_t first = p.a.c.causal ? max(r.len - r.count, 0) : r.len;
    return i * (kRowTileCost + first) * p.a.c.heads + (p.a.c.causal ? i * i * (kRows / 2) : 0);
  }
};

// A stretch of one row tile's tiles.
struct alignas(16) Segment {
  int32_t b, first_tile, end_tile, tiles;   // tiles: of the whole row tile
  int32_t row_tile, row0, rows; // row0: of all rows (token, head); rows: valid ones of 128
  int32_t len, count;           // of the request
  int32_t limit;
  int32_t first;                // 1: of this cluster
  int32_t more;                 // 0: no segment, the ones before it were all
};

struct Control {
  uint64_t k_full[kKSlots], k_empty[kKSlots];   // full: in the leader, both CTAs' bytes
  uint64_t v_full[kVSlots], v_empty[kVSlots];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[2], pv_done[2];         // of the tile's first 64 tokens and the others
  float part[2][4][kHalf];                // [parity][quarter of the tile][row]: maxima, at the end sums
  int64_t warp_sum[kThreads / 32];
  int32_t cut[2][3];                      // begin and end: request, row tile, tile
  Rows rows;                              // of the first request
  Segment segments[kSegments];            // what warp 0 has walked to and not every role has taken
  uint64_t seg_full[kSegments], seg_empty[kSegments];
  uint32_t tmem;
  int abort;
};

constexpr int kOffP = kQBytes, kOffK = kOffP + kPBytes, kOffV = kOffK + kKSlots * kKSlotBytes;
constexpr int kOffControl = kOffV + kVSlots * kVSlotBytes;
constexpr int kSmemBytes = kOffControl + sizeof(Control);
static_assert(kSmemBytes <= kMaxSmemBytes, "shared memory");

// Where cost y of a request lies: row tile and tile.
__device__ __noinline__ void find_cut(const AttendKernelParams& p, const Rows& r, int64_t y, int32_t* cut) {
  // the last row tile whose cost is at most y: near the root of cost(i) = y, then to
  // the right of it (a float's error is far below a row tile but for millions of them)
  const float slope = static_cast<float>(r.cost(p, 1)) - (p.a.c.causal ? kRows / 2 : 0), fy = static_cast<float>(y);
  const float near = p.a.c.causal ? 2.f * fy / (slope + sqrtf(fmaf(slope, slope, 2.f * kRows * fy))) : fy / slope;
  int32_t i = min(max(static_cast<int32_t>(near), 0), r.row_tiles - 1);
  while (i > 0 && r.cost(p, i) > y) --i;
  while (i + 1 < r.row_tiles && r.cost(p, i + 1) <= y) ++i;
  const int64_t from = r.cost(p, i), to = r.cost(p, i + 1);
  const int32_t tiles = r.tiles(p, i);
  cut[0] = i;
  cut[1] = min(static_cast<int32_t>(tiles * (static_cast<float>(y - from) / static_cast<float>(to - from))), max(tiles - 1, 0));
}

// The segments between a cluster's cuts, in order, walked by warp 0 of each CTA.  The
// other roles take them from shared memory: walked by each of them, the code alone
// (cold each time, behind a row tile's loop) held up a row tile by 1.3 us and more.
struct Walk {
  int32_t b, i, k, first;
  Rows r;                       // of request `of`
  int32_t of;
  __device__ __forceinline__ Walk(const int32_t* begin, const Rows& rows)
      : b(begin[0]), i(begin[1]), k(begin[2]), first(1), r(rows), of(begin[0]) {}
};
__device__ __noinline__ bool next_segment(const AttendKernelParams& p, const int32_t* end, Walk* w, Segment* s) {
  while (w->b < end[0] || (w->b == end[0] && (w->i < end[1] || (w->i == end[1] && w->k < end[2])))) {
    if (w->of != w->b) {
      w->r = Rows(p, w->b);
      w->of = w->b;
    }
    const Rows& r = w->r;
    if (w->i >= r.row_tiles) {
      ++w->b;
      w->i = w->k = 0;
      continue;
    }
    const bool last = w->b == end[0] && w->i == end[1];
    const int32_t tiles = r.tiles(p, w->i), local = w->i * kRows;
    *s = Segment{w->b, w->k, last ? end[2] : tiles, tiles, w->i, r.r.first * p.a.c.heads + local,
                 min(kRows, r.rows - local), r.r.len, r.r.count, r.limit, w->first, 1};
    w->first = 0;
    ++w->i;
    w->k = 0;
    if (last) w->b = end[0] + 1;          // that was all
    return true;
  }
  return false;
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void st_global_32(void* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

struct Maps {
  CUtensorMap q, k, v, gather;  // boxes of queries, K, V, and one row high
};

__device__ __forceinline__ uint8_t* shared_base() {
  extern __shared__ __align__(1024) uint8_t smem[];
  return smem;
}
__device__ __forceinline__ Control* control() { return reinterpret_cast<Control*>(shared_base() + kOffControl); }

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
  return mbar_test(bar, parity) || wait_on(bar, parity, &control()->abort, status);
}

// One box of a slot, a lane for each: filled as soon as its slot is free.  first: of
// the slot's lanes the one that announces (in the leader) what both CTAs will write;
// copy: whether this lane has a box of its own.  Warp-wide.
struct Box {
  bool todo, first, copy;
  uint64_t *full, *empty;
  uint32_t full_addr;           // of the leader's
  uint8_t* dst;
  int32_t row, chunk;
};
__device__ __forceinline__ bool load_boxes(Box b, const CUtensorMap* map, uint32_t bytes, uint32_t use, bool leader,
                                           uint32_t* status) {
  for (uint32_t n = 1; __any_sync(0xffffffffu, b.todo); ++n) {
    if (b.todo && (use == 0 || mbar_poll(b.empty, (use - 1) & 1))) {
      if (b.first && leader) mbar_arrive_expect_tx(b.full, 2 * bytes);
      if (b.copy) pair_tma_load_3d(b.dst, map, b.full_addr, 0, b.row, b.chunk);
      b.todo = false;
    }
    if ((n & 1023u) == 0) {     // the slowest of them, with a limit
      bool ok = true;
      if (b.todo) ok = wait_on(b.empty, (use - 1) & 1, &control()->abort, status);
      if (!__all_sync(0xffffffffu, ok)) return false;
    }
  }
  return true;
}

// The lanes whose bit `x` is not set give `hi` for their partner's `lo`.
__device__ __forceinline__ void exchange(uint32_t lo[8], uint32_t hi[8], int x) {
  const bool upper = threadIdx.x & x;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? lo[k] : hi[k], x);
    (upper ? lo[k] : hi[k]) = got;
  }
}

// The next segment for this warp, which says so; false behind the last one and, with
// `ok` false, once a wait gave up.
__device__ __forceinline__ bool take(uint32_t* turn, Segment* s, bool* ok, uint32_t* status) {
  Control* const ctl = control();
  const uint32_t at = *turn % kSegments, parity = (*turn / kSegments) & 1;
  *ok = __all_sync(0xffffffffu, wait(&ctl->seg_full[at], parity, status));
  if (!*ok) return false;
  *s = ctl->segments[at];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&ctl->seg_empty[at]);
  ++*turn;
  return s->more != 0;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_chunk_attend_kernel(const __grid_constant__ AttendKernelParams p, const __grid_constant__ Maps maps) {
  uint8_t* const smem = shared_base();
  Control* const ctl = control();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(&ctl->k_full[i], 1);
      mbar_init(&ctl->k_empty[i], 1);
    }
    for (int i = 0; i < kVSlots; ++i) {
      mbar_init(&ctl->v_full[i], 1);
      mbar_init(&ctl->v_empty[i], 1);
    }
    mbar_init(&ctl->q_full, 1);
    mbar_init(&ctl->q_empty, 1);
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(&ctl->seg_full[i], 1);
      mbar_init(&ctl->seg_empty[i], kSoftmaxWarps + (rank == 0 ? 3 : 1));   // the leader's MMAs too
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->s_free[i], 2 * kSoftmaxWarps);
    }
    mbar_init(&ctl->p_full[0], 2 * kSoftmaxWarps);
    mbar_init(&ctl->p_full[1], kSoftmaxWarps);
    mbar_init(&ctl->pv_done[0], 1);
    mbar_init(&ctl->pv_done[1], 1);
    ctl->abort = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
    prefetch_tmap(&maps.gather);
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
    const int side = threadIdx.x / kSide, t = threadIdx.x % kSide;
    const int32_t batch = p.a.c.batch, each = (batch + kSide - 1) / kSide;
    const int32_t lo = min(t * each, batch), hi = min(lo + each, batch);
    int64_t sum = 0;
    bool bad = false;
    Rows r;
    for (int32_t b = hi; b-- > lo;) {     // down, so that r ends as the first one's
      r = Rows(p, b);
      bad |= r.r.bad || r.limit < r.r.len;
      sum += r.cost(p, r.row_tiles);
    }
    if (bad && blockIdx.x == 0 && p.a.c.status) atomicOr(p.a.c.status, MLA_STATUS_BAD_INDEX);
    int64_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) ctl->warp_sum[warp] = upto;
    if (t == 0) {                         // a cut at the end of the work lies in no request
      ctl->cut[side][0] = batch;
      ctl->cut[side][1] = ctl->cut[side][2] = 0;
    }
    __syncthreads();
    int64_t at = upto - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kSide / 32; ++w) {
      const int64_t of = ctl->warp_sum[side * (kSide / 32) + w];
      if (w < t / 32) at += of;
      total += of;
    }
    // the same for both sides of a cut, and not descending: that is all it has to be
    const int c = cluster + side;
    const float share = static_cast<float>(total) * (static_cast<float>(c) / static_cast<float>(clusters));
    const int64_t x = c == clusters ? total : min(static_cast<int64_t>(share), total);
    if (at <= x && x < at + sum) {
      int32_t b = lo;
      int64_t cost = r.cost(p, r.row_tiles);
      while (x >= at + cost) {
        at += cost;
        r = Rows(p, ++b);
        cost = r.cost(p, r.row_tiles);
      }
      ctl->cut[side][0] = b;
      if (side == 0) ctl->rows = r;
      find_cut(p, r, x - at, ctl->cut[side] + 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();           // both CTAs have their half of tensor memory
  tc_fence_after();

  const uint32_t tmem = ctl->tmem;
  uint32_t* const status = p.a.c.status;
  const int32_t* const end = ctl->cut[1];
  Segment s;
  uint32_t turn = 0;            // segments walked to, or taken
  bool ok = true;

  if (warp == 0) {
    // queries and K: this CTA's 64 rows, and its 64 tokens of every tile
    const uint32_t q_bar = mapa_shared(smem_u32(&ctl->q_full), 0), k_bar = mapa_shared(smem_u32(ctl->k_full), 0);
    const int pieces = kHalf / p.box_rows, boxes = pieces == 1 ? 1 : kKChunks * pieces;   // of a slot
    const int slots_at_once = min(kKSlots, 32 / boxes);
    Walk walk(ctl->cut[0], ctl->rows);
    uint32_t use = 0, nq = 0;
    for (;; ++turn) {
      if (!next_segment(p, end, &walk, &s)) s.more = 0;
      const uint32_t at = turn % kSegments;
      ok = __all_sync(0xffffffffu, ok && (turn < kSegments || wait(&ctl->seg_empty[at], (turn / kSegments - 1) & 1, status)));
      if (!ok) break;
      if (lane == 0) {
        ctl->segments[at] = s;
        mbar_arrive(&ctl->seg_full[at]);
      }
      if (!s.more) break;
      if (s.end_tile <= s.first_tile) continue;
      TilePages pages;
      pages.load(p.a.c, s.b, s.limit, s.first_tile, lane);
      const int32_t dense = p.dense ? p.dense[s.b].x : -1;
      ok = nq == 0 || wait(&ctl->q_empty, (nq - 1) & 1, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      ++nq;
      if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&ctl->q_full, 2 * kQBytes);
      if (lane < kChunks / kKChunks)
        pair_tma_load_3d(smem + lane * kKSlotBytes, &maps.q, q_bar, 0, s.row0 + kHalf * static_cast<int32_t>(rank), kKChunks * lane);
#pragma unroll 1
      for (int32_t tile = s.first_tile; ok && tile < s.end_tile; ++tile, ++use) {
        const TileRows rows(p.a.c, s.limit, tile, pages, dense, lane);
        if (pages.bad(p.a.c) && rank == 0 && lane == 0 && status) atomicOr(status, MLA_STATUS_BAD_PAGE);
        if (tile + 1 < s.end_tile) pages.load(p.a.c, s.b, s.limit, tile + 1, lane);
        // boxes of 64 tokens and the slot's chunks, or of a smaller page and one chunk.
        // Slots that hold no row are read all the same, pages that are not there from
        // the pool's start: their scores are masked out.
        for (int j0 = 0; ok && j0 < kKSlots; j0 += slots_at_once) {
          const int j = j0 + lane / boxes, i = lane % boxes, piece = i & (pieces - 1), chunk = i / pieces;
          const int piece_at = 4 * static_cast<int>(rank) + piece * (p.box_rows >> 4);
          int32_t row = max(__shfl_sync(0xffffffffu, rows.base, piece_at), 0);
          if (p.dense) row = dense + tile * kTok + 16 * piece_at;   // whole tiles side by side, whatever the pages
          const bool todo = lane < slots_at_once * boxes && j < kKSlots;
          ok = load_boxes(Box{todo, i == 0, true, &ctl->k_full[j], &ctl->k_empty[j], k_bar + 8 * j,
                              smem + kOffK + j * kKSlotBytes + chunk * kChunkBytes + piece * p.box_rows * 128, row,
                              kKChunks * j + chunk},
                          &maps.k, kKSlotBytes, use, rank == 0, status);
        }
      }
    }
  } else if (warp == 3) {
    // V: this CTA's 256 latent columns of every token of the tile
    const uint32_t v_bar = mapa_shared(smem_u32(ctl->v_full), 0);
    const int v_rows = min(p.box_rows, kVTokens), pieces = kVTokens / v_rows;
    uint32_t use = 0;
    while (ok && take(&turn, &s, &ok, status)) {
      if (s.end_tile <= s.first_tile) continue;
      TilePages pages;
      pages.load(p.a.c, s.b, s.limit, s.first_tile, lane);
      const int32_t dense = p.dense ? p.dense[s.b].x : -1;
#pragma unroll 1
      for (int32_t tile = s.first_tile; ok && tile < s.end_tile; ++tile, ++use) {
        const TileRows rows(p.a.c, s.limit, tile, pages, dense, lane);
        if (tile + 1 < s.end_tile) pages.load(p.a.c, s.b, s.limit, tile + 1, lane);
        // pieces of 32 tokens, or of a smaller page.  What no row stands in is zeros (its
        // weight is zero, and nothing else must come of the product): pieces without
        // any row are read behind the tensor's end, which fills with zeros
        const int g = lane / pieces, piece = lane % pieces, t = kVTokens * g + v_rows * piece;
        const int32_t base = __shfl_sync(0xffffffffu, rows.base, (t >> 4) & 7);
        const bool todo = lane < kVSlots * pieces, none = base < 0, whole = !none && rows.left - t >= v_rows;
        const uint32_t part = __ballot_sync(0xffffffffu, todo && !none && !whole);
        ok = load_boxes(Box{todo, piece == 0, none || whole, &ctl->v_full[g], &ctl->v_empty[g], v_bar + 8 * g,
                            smem + kOffV + g * kVSlotBytes + piece * (kVSlotBytes / 2), whole ? base : p.map_rows,
                            4 * static_cast<int>(rank)},
                        &maps.v, kVSlotBytes, use, rank == 0, status);
        // the piece of the last token row by row, in gathers of four
        if (ok && part) {
          const int from = __ffs(part) - 1, groups = v_rows / 4, atom = lane / groups, group = lane % groups;
          int32_t four[4];
          rows.four((kVTokens * (from / pieces) + v_rows * (from % pieces) + 4 * group) & (kTok - 1), four);
          if (lane < v_rows)
            pair_tma_gather4(smem + kOffV + (from / pieces) * kVSlotBytes + (from % pieces) * (kVSlotBytes / 2) +
                                 atom * v_rows * 128 + group * 512,
                             &maps.gather, v_bar + 8 * (from / pieces), (4 * rank + atom) * kChunkElems, four);
        }
      }
    }
  } else if (warp == 1) {
    // The pair's MMAs go out from two warps, S from this one and O from warp 2, so that
    // one's run while the other waits.
    if (rank == 0) {
      const uint32_t idesc = make_idesc_bf16(kRows, kTok, false, false);
      const MatrixWords q0(smem, 16, 1024), k0(smem + kOffK, 16, 1024);
      uint32_t use = 0, nq = 0;
      while (ok && take(&turn, &s, &ok, status)) {
        if (s.end_tile <= s.first_tile) continue;
        ok = __all_sync(0xffffffffu, wait(&ctl->q_full, nq++ & 1, status));
#pragma unroll 1
        for (int32_t tile = s.first_tile; ok && tile < s.end_tile; ++tile, ++use) {
          const uint32_t col = tmem + kColS + 64 * (use & 1);
          ok = use < 2 || __all_sync(0xffffffffu, wait(&ctl->s_free[use & 1], ((use >> 1) - 1) & 1, status));
#pragma unroll 1
          for (int j = 0; ok && j < kKSlots; ++j) {
            ok = __all_sync(0xffffffffu, wait(&ctl->k_full[j], use & 1, status));
            tc_fence_after();
            const uint32_t at = (j * kKSlotBytes) >> 4;
#pragma unroll
            for (int m = 0; m < 4 * kKChunks; ++m) {
              const uint32_t o = at + (((m >> 2) * kChunkBytes + (m & 3) * 32) >> 4);
              pair_mma_bf16(col, q0.lo + o, q0.hi, k0.lo + o, k0.hi, idesc, j > 0 || m > 0);
            }
            pair_commit(&ctl->k_empty[j]);
          }
          pair_commit(&ctl->s_full[use & 1]);
        }
        pair_commit(&ctl->q_empty);
      }
    }
  } else if (warp == 2) {
    if (rank == 0) {
      const uint32_t idesc = make_idesc_bf16(kRows, 256, false, true);
      const int v_rows = min(p.box_rows, kVTokens), v_atom = v_rows * 128;
      const MatrixWords p0(smem + kOffP, 16, 1024), v0(smem + kOffV, v_atom, 1024);
      const uint32_t v_step = (v_rows == kVTokens ? 2048 : kVSlotBytes / 2) >> 4;   // to the slot's second 16 tokens
      const uint32_t v_half = (2 * v_atom) >> 4;                                    // to the second 128 columns
      uint32_t use = 0;
      while (ok && take(&turn, &s, &ok, status)) {
#pragma unroll 1
        for (int32_t tile = s.first_tile; ok && tile < s.end_tile; ++tile, ++use) {
#pragma unroll 1
          for (int g = 0; ok && g < kVSlots; ++g) {
            if ((g & 1) == 0) ok = __all_sync(0xffffffffu, wait(&ctl->p_full[g >> 1], use & 1, status));
            if (!ok) break;
            ok = __all_sync(0xffffffffu, wait(&ctl->v_full[g], use & 1, status));
            tc_fence_after();
            const uint32_t vb = v0.lo + ((g * kVSlotBytes) >> 4);
            const uint32_t pa = p0.lo + (((g >> 1) * kChunkBytes + (g & 1) * 64) >> 4);
#pragma unroll
            for (int m = 0; m < 4; ++m) {   // 16 tokens m & 1, columns 128 (m >> 1) .. of each CTA's 256
              pair_mma_bf16(tmem + kColO + 128 * (m >> 1), pa + 2 * (m & 1), p0.hi,
                            vb + (m & 1) * v_step + (m >> 1) * v_half, v0.hi, idesc,
                            tile > s.first_tile || g > 0 || (m & 1));
            }
            pair_commit(&ctl->v_empty[g]);
            if (g & 1) pair_commit(&ctl->pv_done[g >> 1]);
          }
        }
      }
    }
  } else {
    // softmax: lane l of tensor memory is row l % 64, tokens 64 (l / 64) .. of which
    // the warps 4 .. 7 take the first 32 and 8 .. 11 the others
    const int quad = warp & 3, l = quad * 32 + lane, row = l & 63, half = l >> 6, side = (warp >> 2) - 1;
    const int quarter = 2 * half + side;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t p_bar = mapa_shared(smem_u32(ctl->p_full), 0), s_bar = mapa_shared(smem_u32(ctl->s_free), 0);
    const uint32_t row_bar = 1 + (quad & 1);   // the 128 threads of 32 rows
    uint8_t* const prow = smem + kOffP + half * kChunkBytes + row * 128;
    const float scale = p.a.c.scale_log2;
    uint32_t use = 0;
    int slots_used = 0;
    bool failed = false;
    Segment next;
    bool more = take(&turn, &next, &ok, status);
    // a wait that gave up is agreed on at the next barrier of the row's warps
    if (named_bar_or(row_bar, 128, !ok)) more = false;
    while (more) {
      s = next;
      const int n = s.end_tile - s.first_tile;
      const int32_t at = kHalf * static_cast<int32_t>(rank) + row;   // of the row tile
      const bool valid = at < s.rows;
      const ChunkRequest request(s.len, s.count);
      const int32_t seen = valid ? min(request.seen((s.row_tile * kRows + at) / p.a.c.heads, p.a.c.causal), s.limit) : 0;
      float ref = -INFINITY, sum = 0.f, sum_rounded = 0.f;
      TilePages pages;
      if (n > 0) pages.load(p.a.c, s.b, s.limit, s.first_tile, lane);
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++use) {
        const uint32_t bad = (pages.bad(p.a.c) >> (2 * quarter)) & 3u;
        if (i + 1 < n) pages.load(p.a.c, s.b, s.limit, s.first_tile + i + 1, lane);
        const int32_t vis = min(max(seen - (s.first_tile + i) * kTok - 32 * quarter, 0), 32);
        failed |= !__all_sync(0xffffffffu, wait(&ctl->s_full[use & 1], (use >> 1) & 1, status));
        tc_fence_after();
        uint32_t x[32];
        tmem_ld32(tmem + lanes + kColS + 64 * (use & 1) + 32 * side, x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cluster_mbar_arrive(s_bar + 8 * (use & 1));
        if (vis < 32 || bad) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (k >= vis || (bad >> (k >> 4) & 1)) x[k] = 0xFF800000u;   // -inf
        }
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};   // chains that run side by side
#pragma unroll
        for (int k = 0; k < 32; k += 2)
          tops[(k >> 1) & 3] = max3(tops[(k >> 1) & 3], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
        float* const part = &ctl->part[use & 1][0][row];
        part[kHalf * quarter] = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
        if (named_bar_or(row_bar, 128, failed)) break;
        const float top = fmaxf(max3(part[0], part[kHalf], part[2 * kHalf]), part[3 * kHalf]) * scale;
        float grow_by = 1.f;
        if (top > ref + 8.f) {   // from -inf at once
          grow_by = exp2_approx(ref - top);
          ref = top;
          sum *= grow_by;
          sum_rounded *= grow_by;
        }
        const float base = ref == -INFINITY ? 0.f : ref;
        const float2 scale2 = make_float2(scale, scale), base2 = make_float2(-base, -base);
        uint32_t w[16];
        float2 sums[2] = {}, rounded[2] = {};
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float2 e = __ffma2_rn(make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), scale2, base2);
          e.x = exp2_approx(e.x);
          e.y = exp2_approx(e.y);
          w[k] = pack_bf16(e);            // V's type; what it costs stands at the top
          sums[k & 1] = __fadd2_rn(sums[k & 1], e);
          rounded[k & 1] = __fadd2_rn(rounded[k & 1], make_float2(bf16_lo(w[k]), bf16_hi(w[k])));
        }
        sum += (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
        sum_rounded += (rounded[0].x + rounded[0].y) + (rounded[1].x + rounded[1].y);
        // P's half is written when the last tile's product has read it.  The first half's
        // product starts on its own: it also waits for the other half's warps to say that
        // their lanes of O are ready, once the last tile's first product is through
        if (use > 0) failed |= !__all_sync(0xffffffffu, wait(&ctl->pv_done[0], (use - 1) & 1, status));
        if (i > 0 && __any_sync(0xffffffffu, grow_by != 1.f)) {   // rare: 8 more bits than any tile before
          failed |= !__all_sync(0xffffffffu, wait(&ctl->pv_done[1], (use - 1) & 1, status));
          tc_fence_after();
#pragma unroll 1
          for (int c = 128 * side; c < 128 * side + 128; c += 16) {
            uint32_t o[16];
            tmem_ld16(tmem + lanes + kColO + c, o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * grow_by);
            tmem_st16(tmem + lanes + kColO + c, o);
          }
          tc_fence_before();
          __syncwarp();
        }
        if (half == 1) {
          if (lane == 0) cluster_mbar_arrive(p_bar);
          if (use > 0) failed |= !__all_sync(0xffffffffu, wait(&ctl->pv_done[1], (use - 1) & 1, status));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(prow + (((4 * side + k) ^ (row & 7)) << 4)) =
              make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) cluster_mbar_arrive(p_bar + 8 * half);
      }
      more = take(&turn, &next, &ok, status);   // while the last product runs
      failed |= !ok;
      // the row's output: whole, or this cluster's part of it
      if (n > 0) {
        if (named_bar_or(row_bar, 128, failed)) break;   // the maxima have been read
        ctl->part[0][quarter][row] = sum_rounded;
        ctl->part[1][quarter][row] = sum;
        failed |= !__all_sync(0xffffffffu, wait(&ctl->pv_done[1], (use - 1) & 1, status));
        if (named_bar_or(row_bar, 128, failed)) break;
        sum_rounded = sum = 0.f;
        for (int k = 0; k < 4; ++k) {
          sum_rounded += ctl->part[0][k][row];
          sum += ctl->part[1][k][row];
        }
        tc_fence_after();
      }
      const float inv = sum_rounded > 0.f || sum_rounded != sum_rounded ? 1.f / sum_rounded : 0.f;
      const bool whole = s.first_tile == 0 && s.end_tile == s.tiles, none = sum == 0.f;   // none: O may hold anything
      const int slot = 2 * cluster + (s.first ? 0 : 1);
      if (!whole) {
        slots_used |= s.first ? 1 : 2;
        if (rank == 0 && threadIdx.x == 128)
          p.segments[slot] = make_int4(s.first_tile == 0 ? kOpens : kContinues, s.row0, s.rows, 0);
      }
      // 64 columns of a row at a time.  Parts go out as they are (ChunkWorkspace's layout
      // puts the lanes' 32 bytes side by side); of whole rows' bf16 four lanes exchange
      // their 32-byte pieces first, so that a store writes 128 bytes of each of 8 rows
#pragma unroll 1
      for (int c = 128 * side; c < 128 * side + 128; c += 64) {
        uint32_t w[4][8];
        const int col = 256 * half + c;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t o[32] = {};
          if (n > 0) tmem_ld32(tmem + lanes + kColO + c + 32 * h, o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = none ? 0u : __float_as_uint(__uint_as_float(o[k]) * inv);
          if (!whole) {
            float* out = p.part_o + static_cast<int64_t>(slot) * kRows * kDc + ((col + 32 * h) * kRows + 8 * at);
            if (valid) {
#pragma unroll
              for (int k = 0; k < 4; ++k) st_global_32(out + 8 * k * kRows, o + 8 * k);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              w[2 * h + (k >> 3)][k & 7] = pack_bf16(make_float2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])));
          }
        }
        if (whole) {
          exchange(w[0], w[1], 1);
          exchange(w[2], w[3], 1);
          exchange(w[0], w[2], 2);
          exchange(w[1], w[3], 2);
          const int32_t row0 = at & ~3;
          uint16_t* out = p.a.o + static_cast<int64_t>(s.row0 + row0) * kDc + col + 16 * (lane & 3);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (row0 + k < s.rows) st_global_32(out + k * kDc, w[k]);
        }
        __syncwarp();
      }
      if (valid && quarter == 0)
        (whole ? p.a.lse[s.row0 + at] : p.part_lse[slot * kRows + at]) =
            none ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
      tc_fence_before();
      if (named_bar_or(row_bar, 128, failed)) break;   // the sums have been read
    }
    if (rank == 0 && threadIdx.x == 128) {
      const bool idle = ctl->cut[0][0] == end[0] && ctl->cut[0][1] == end[1] && ctl->cut[0][2] == end[2];
      if (!(slots_used & 1)) p.segments[2 * cluster] = make_int4(idle ? kIdle : kNone, 0, 0, 0);
      if (!(slots_used & 2)) p.segments[2 * cluster + 1] = make_int4(kNone, 0, 0, 0);
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

// The merge of row tiles that were cut: lse = ln sum exp(lse_i), o = sum
// exp(lse_i - lse) o_i over the parts in order.  Block (slot, 8 rows); the slot that
// opens a row tile looks for the clusters that continue it.  Bound by the latency of
// segments, lse and parts one after another: behind the attention it adds 2 to 5 us.
constexpr int kMergeWarps = 8;
constexpr int kMaxParts = kMaxChunkClusters + 1;

__global__ void __launch_bounds__(32 * kMergeWarps) mla_chunk_merge_kernel(const __grid_constant__ AttendKernelParams p, int clusters) {
  __shared__ int parts[kMaxParts], s_count;
  __shared__ float weight[kMaxParts * kMergeWarps], s_inv[kMergeWarps];
  after_predecessor();
  const int slot = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 none = make_int4(kNone, 0, 0, 0), own = p.segments[slot];
  // with it, ahead of its use, what the next 32 clusters open with
  int4 next = slot / 2 + 1 + lane < clusters && warp == 0 ? p.segments[2 * (slot / 2 + 1 + lane)] : none;
  const int r = blockIdx.y * kMergeWarps + warp;
  if (own.x != kOpens || static_cast<int>(blockIdx.y) * kMergeWarps >= own.z) return;
  // the parts in order: this slot, and the first ones of the clusters behind it that
  // continue the row tile (idle ones between them have none)
  if (warp == 0) {
    int count = 1;
    if (lane == 0) parts[0] = slot;
    for (int base = slot / 2 + 1; base < clusters; base += 32) {
      const int c = base + lane;
      const int4 s = next;
      next = c + 32 < clusters ? p.segments[2 * (c + 32)] : none;
      const bool part = s.x == kContinues && s.y == own.y, stop = !part && s.x != kIdle;
      const uint32_t stops = __ballot_sync(0xffffffffu, stop);
      const uint32_t before = stops ? (1u << (__ffs(stops) - 1)) - 1u : 0xffffffffu;
      const uint32_t found = __ballot_sync(0xffffffffu, part) & before;
      if (found >> lane & 1) parts[count + __popc(found & ((1u << lane) - 1u))] = 2 * c;
      count += __popc(found);
      if (stops) break;
    }
    if (lane == 0) s_count = count;
  }
  __syncthreads();
  const int count = s_count;
  // a warp for a row's weights
  const bool valid = r < own.z;
  float top = -INFINITY, sum = 0.f;
  for (int i = lane; i < count; i += 32)
    if (valid) top = fmaxf(top, p.part_lse[parts[i] * kRows + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  for (int i = lane; i < count; i += 32) {
    const float part = valid ? p.part_lse[parts[i] * kRows + r] : -INFINITY;
    const float e = part == -INFINITY ? 0.f : expf(part - top);
    weight[i * kMergeWarps + warp] = e;
    sum += e;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int64_t row0 = own.y + static_cast<int64_t>(blockIdx.y) * kMergeWarps;
  if (lane == 0) {
    s_inv[warp] = top == -INFINITY ? 0.f : 1.f / sum;
    if (valid) p.a.lse[row0 + warp] = top == -INFINITY ? -INFINITY : top + logf(sum);
  }
  __syncthreads();
  // and for 64 columns of all rows: 4 of a row's a lane, two groups of eight at once
  const int row = (lane >> 1) & 7, group = 8 * warp + (lane >> 4);
  if (static_cast<int>(blockIdx.y) * kMergeWarps + row >= own.z) return;
  const float* const from = p.part_o + (group * kRows + static_cast<int>(blockIdx.y) * kMergeWarps + row) * 8 + 4 * (lane & 1);
  float4 acc[4] = {};
#pragma unroll 4
  for (int i = 0; i < count; ++i) {
    const float* o = from + static_cast<int64_t>(parts[i]) * kRows * kDc;
    const float e = weight[i * kMergeWarps + row];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(o + 2 * k * 8 * kRows);
      acc[k].x = fmaf(e, v.x, acc[k].x);
      acc[k].y = fmaf(e, v.y, acc[k].y);
      acc[k].z = fmaf(e, v.z, acc[k].z);
      acc[k].w = fmaf(e, v.w, acc[k].w);
    }
  }
  const float inv = s_inv[row];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    *reinterpret_cast<uint2*>(p.a.o + (row0 + row) * kDc + 8 * (group + 2 * k) + 4 * (lane & 1)) =
        make_uint2(pack_bf16(make_float2(acc[k].x * inv, acc[k].y * inv)), pack_bf16(make_float2(acc[k].z * inv, acc[k].w * inv)));
}

}  // namespace

cudaError_t launch_chunk_attend(const AttendParams& a, const ChunkWorkspace& w, cudaStream_t stream) {
  AttendKernelParams p;
  p.a = a;
  p.part_o = w.part_o;
  p.part_lse = w.part_lse;
  p.segments = reinterpret_cast<int4*>(w.segments);
  p.dense = w.starts;
  p.box_rows = w.starts ? kHalf : a.c.page_shift > 6 ? kHalf : 1 << a.c.page_shift;
  const void* rows = w.starts ? static_cast<const void*>(w.rows) : a.c.kv;
  const uint64_t count = w.starts ? static_cast<uint64_t>(w.capacity > 0 ? w.capacity : 1) : static_cast<uint64_t>(a.c.num_pages) << a.c.page_shift;
  p.map_rows = static_cast<int32_t>(count);
  Maps maps;
  if (!make_map_chunks_bf16(&maps.q, a.c.q, kDqk, static_cast<uint64_t>(a.c.tokens) * a.c.heads, kDqk * 2, kHalf, kKChunks) ||
      !make_map_chunks_bf16(&maps.k, rows, kDqk, count, kDqk * 2, p.box_rows, p.box_rows == kHalf ? kKChunks : 1) ||
      !make_map_chunks_bf16(&maps.v, rows, kDqk, count, kDqk * 2, p.box_rows < 32 ? p.box_rows : 32, 4) ||
      !make_map_bf16(&maps.gather, rows, kDqk, count, kDqk * 2, kChunkElems, 1))
    return cudaErrorInvalidValue;
  cudaError_t err = set_smem_attr_once(reinterpret_cast<const void*>(mla_chunk_attend_kernel), kSmemAttrChunk, kSmemBytes);
  if (err != cudaSuccess) return err;
  err = launch_dependent(mla_chunk_attend_kernel, dim3(2 * w.clusters), kThreads, kSmemBytes, stream, p, maps);
  if (err != cudaSuccess) return err;
  return launch_dependent(mla_chunk_merge_kernel, dim3(2 * w.clusters, kRows / kMergeWarps), 32 * kMergeWarps, 0, stream, p, w.clusters);
}

}  // namespace mla
