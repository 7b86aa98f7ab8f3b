// Host side of include/mla_chunk.h: argument checks, plans and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "mla_chunk_internal.h"

using namespace mla;

namespace {

constexpr int32_t kChunkPlanMark = 0x43484B31, kEvictPlanMark = 0x45564331;
constexpr int64_t kAlign = 256;
constexpr int32_t kRowsOfTile = 128;   // rows (token, head) that a pair of CTAs takes at a time

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int64_t align_up(int64_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
int shift_of(int32_t page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }
int64_t row_bytes(int32_t kv) {
  return kv == MLA_KV_BF16 ? kDqk * 2 : kv == MLA_KV_FP8_E4M3_E8M0 ? kFp8RowBytes : kFp4RowBytes;
}

// Whether two arrays of `bytes` each share memory.
bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + static_cast<uintptr_t>(b_bytes) && y < x + static_cast<uintptr_t>(a_bytes);
}

struct Array {
  const void* base;
  int64_t bytes;
  const void* own;   // of one that is written: the input that it may be
};
// Whether every array that is written stands alone, but for an output that is its input.
bool stand_alone(const Array* written, int n_written, const Array* read, int n_read) {
  for (int i = 0; i < n_written; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(written[i].base, written[i].bytes, written[j].base, written[j].bytes)) return false;
    for (int j = 0; j < n_read; ++j)
      if (!(written[i].own == read[j].base && written[i].base == read[j].base) &&
          overlap(written[i].base, written[i].bytes, read[j].base, read[j].bytes))
        return false;
  }
  return true;
}
template <int kWritten, int kRead>
bool stand_alone(const Array (&written)[kWritten], const Array (&read)[kRead]) {
  return stand_alone(written, kWritten, read, kRead);
}

int64_t cache_bytes(const mla_problem& pr) { return static_cast<int64_t>(pr.num_pages) * pr.page_size * row_bytes(pr.kv_dtype); }
// Of [batch][stride] entries of 4 bytes: to the last request's last slot.
int64_t entry_bytes(const mla_problem& pr, int64_t stride) {
  const int64_t slots = static_cast<int64_t>(pr.max_pages_per_seq) * pr.page_size;
  return ((pr.batch - 1) * stride + (stride < slots ? stride : slots)) * 4;
}
int64_t table_bytes(const mla_problem& pr) { return static_cast<int64_t>(pr.batch) * pr.max_pages_per_seq * 4; }

int check_chunk_problem(const mla_problem* pr) {
  const int rc = check_cache_shape(pr);
  if (rc != MLA_OK) return rc;
  if (pr->num_heads < 1 || !(pr->causal == 0 || pr->causal == 1) || !std::isfinite(pr->sm_scale) ||
      pr->sm_scale <= 0.f)
    return MLA_ERR_INVALID_ARGUMENT;
  if (pr->num_heads > MLA_CHUNK_MAX_HEADS || pr->batch > MLA_CHUNK_MAX_REQUESTS || pr->topk_width != 0)
    return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

// What the attention and the weights check alike.
int fill_chunk(const mla_chunk_plan* plan, const void* q, const int32_t* starts, const void* kv,
               const int32_t* block_table, const int32_t* lens, const void* workspace,
               size_t workspace_bytes, uint32_t* status, ChunkParams* p) {
  if (plan == nullptr || plan->mark != kChunkPlanMark) return MLA_ERR_INVALID_ARGUMENT;
  const mla_problem& pr = plan->problem;
  const int rc = check_chunk_problem(&pr);
  if (rc != MLA_OK) return rc;
  if (q == nullptr && plan->tokens == 0) q = workspace;   // no query is read
  if (!q || !starts || !kv || !block_table || !lens || !workspace) return MLA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < static_cast<size_t>(plan->workspace_bytes)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(workspace, 16) || !aligned(starts, 4) ||
      !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(status, 4))
    return MLA_ERR_MISALIGNED;
  p->q = static_cast<const uint16_t*>(q);
  p->starts = starts;
  p->kv = static_cast<const uint8_t*>(kv);
  p->block_table = block_table;
  p->lens = lens;
  p->status = status;
  p->tokens = plan->tokens;
  p->batch = pr.batch;
  p->heads = pr.num_heads;
  p->page_shift = shift_of(pr.page_size);
  p->num_pages = pr.num_pages;
  p->max_pages = pr.max_pages_per_seq;
  p->kv_dtype = pr.kv_dtype;
  p->causal = pr.causal;
  p->scale_log2 = pr.sm_scale * 1.4426950408889634f;
  return MLA_OK;
}

// Expanded rows with each request's padding.
int64_t dense_rows(int64_t context_tokens, int32_t batch) {
  return context_tokens + static_cast<int64_t>(batch) * (kDensePad - 1);
}

ChunkWorkspace workspace_of(const mla_chunk_plan& plan, void* workspace) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool quantised = plan.problem.kv_dtype != MLA_KV_BF16;
  ChunkWorkspace w;
  w.part_o = reinterpret_cast<float*>(ws + plan.ws_partial_o);
  w.part_lse = reinterpret_cast<float*>(ws + plan.ws_partial_lse);
  w.segments = reinterpret_cast<int32_t*>(ws + plan.ws_segments);
  w.starts = quantised ? reinterpret_cast<int2*>(ws + plan.ws_starts) : nullptr;
  w.rows = quantised ? reinterpret_cast<uint16_t*>(ws + plan.ws_rows) : nullptr;
  w.context = static_cast<int32_t>(plan.context_tokens);
  w.capacity = quantised ? static_cast<int32_t>(dense_rows(plan.context_tokens, plan.problem.batch)) : 0;
  w.clusters = plan.clusters;
  return w;
}

}  // namespace

extern "C" {

int mla_chunk_make_plan(const mla_problem* problem, int32_t tokens, int64_t context_tokens,
                        int32_t sm_count, mla_chunk_plan* plan_out, size_t* workspace_bytes) {
  const int rc = check_chunk_problem(problem);
  if (rc != MLA_OK) return rc;
  const bool quantised = problem->kv_dtype != MLA_KV_BF16;
  if (tokens < 0 || sm_count < 1 || plan_out == nullptr || (quantised && context_tokens < 0))
    return MLA_ERR_INVALID_ARGUMENT;
  // rows of queries, and expanded rows, are 32-bit coordinates
  if (static_cast<int64_t>(tokens) * problem->num_heads > INT32_MAX - kRowsOfTile ||
      (quantised && (context_tokens > INT32_MAX || dense_rows(context_tokens, problem->batch) > INT32_MAX - kRowsOfTile)))
    return MLA_ERR_UNSUPPORTED;
  mla_chunk_plan pl;
  std::memset(&pl, 0, sizeof(pl));
  pl.problem = *problem;
  pl.tokens = tokens;
  pl.sm_count = sm_count;
  pl.context_tokens = quantised ? context_tokens : 0;
  pl.clusters = sm_count < 4 ? 1 : sm_count / 2 < kMaxChunkClusters ? sm_count / 2 : kMaxChunkClusters;
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at = align_up(at + bytes);
    return here;
  };
  const int64_t parts = 2 * static_cast<int64_t>(pl.clusters);
  pl.ws_partial_o = take(parts * kRowsOfTile * kDc * 4);
  pl.ws_partial_lse = take(parts * kRowsOfTile * 4);
  pl.ws_segments = take(parts * 16);
  pl.ws_starts = take((static_cast<int64_t>(problem->batch) + 1) * 8);
  pl.ws_rows = take(quantised ? dense_rows(context_tokens, problem->batch) * kDqk * 2 : 0);
  pl.workspace_bytes = at;
  pl.mark = kChunkPlanMark;
  *plan_out = pl;
  if (workspace_bytes) *workspace_bytes = static_cast<size_t>(at);
  return MLA_OK;
}

int mla_chunk_attend(const mla_chunk_plan* plan, const void* q_hat, const int32_t* query_starts,
                     const void* kv_cache, const int32_t* block_table, const int32_t* seq_lens,
                     void* workspace, size_t workspace_bytes, void* o_lat, float* lse,
                     uint32_t* status, mla_stream_t stream) {
  AttendParams p;
  const int rc = fill_chunk(plan, q_hat, query_starts, kv_cache, block_table, seq_lens, workspace,
                            workspace_bytes, status, &p.c);
  if (rc != MLA_OK) return rc;
  if (plan->tokens == 0 || plan->problem.batch == 0) return MLA_OK;
  if (!o_lat || !lse) return MLA_ERR_INVALID_ARGUMENT;
  if (!aligned(o_lat, 32) || !aligned(lse, 4)) return MLA_ERR_MISALIGNED;
  const mla_problem& pr = plan->problem;
  const int64_t rows = static_cast<int64_t>(plan->tokens) * pr.num_heads;
  const Array written[] = {{workspace, plan->workspace_bytes, nullptr}, {o_lat, rows * kDc * 2, nullptr},
                           {lse, rows * 4, nullptr}, {status, 4, nullptr}};
  const Array read[] = {{q_hat, rows * kDqk * 2, nullptr}, {query_starts, pr.batch * 4ll + 4, nullptr},
                        {kv_cache, cache_bytes(pr), nullptr}, {block_table, table_bytes(pr), nullptr},
                        {seq_lens, pr.batch * 4ll, nullptr}};
  if (!stand_alone(written, read)) return MLA_ERR_INVALID_ARGUMENT;
  p.o = static_cast<uint16_t*>(o_lat);
  p.lse = lse;
  const ChunkWorkspace w = workspace_of(*plan, workspace);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (w.starts && launch_expand(p.c, w, st) != cudaSuccess) return MLA_ERR_CUDA;
  return launch_chunk_attend(p, w, st) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_cache_weights(const mla_chunk_plan* plan, const void* q_hat, const float* lse,
                      const int32_t* query_starts, const void* kv_cache,
                      const int32_t* block_table, const int32_t* seq_lens, void* workspace,
                      size_t workspace_bytes, const float* weights_in, float* weights_out,
                      int64_t stride, uint32_t* status, mla_stream_t stream) {
  WeightsParams p;
  const int rc = fill_chunk(plan, q_hat, query_starts, kv_cache, block_table, seq_lens, workspace,
                            workspace_bytes, status, &p.c);
  if (rc != MLA_OK) return rc;
  if ((!lse && plan->tokens > 0) || !weights_out || stride < 1 || stride > INT64_MAX / 8 / (p.c.batch + 1)) return MLA_ERR_INVALID_ARGUMENT;
  if (!aligned(lse, 4) || !aligned(weights_in, 4) || !aligned(weights_out, 4)) return MLA_ERR_MISALIGNED;
  const mla_problem& pr = plan->problem;
  if (pr.batch == 0) return MLA_OK;
  const int64_t bytes = entry_bytes(pr, stride), rows = static_cast<int64_t>(plan->tokens) * pr.num_heads;
  const Array written[] = {{workspace, plan->workspace_bytes, nullptr}, {weights_out, bytes, weights_in}, {status, 4, nullptr}};
  const Array read[] = {{q_hat, rows * kDqk * 2, nullptr}, {lse, rows * 4, nullptr},
                        {query_starts, pr.batch * 4ll + 4, nullptr}, {kv_cache, cache_bytes(pr), nullptr},
                        {block_table, table_bytes(pr), nullptr}, {seq_lens, pr.batch * 4ll, nullptr},
                        {weights_in, bytes, nullptr}};
  if (!stand_alone(written, read)) return MLA_ERR_INVALID_ARGUMENT;
  p.lse = lse;
  p.in = weights_in;
  p.out = weights_out;
  p.stride = stride;
  const ChunkWorkspace w = workspace_of(*plan, workspace);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (w.starts && launch_expand(p.c, w, st) != cudaSuccess) return MLA_ERR_CUDA;
  return launch_cache_weights(p, w, st) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_evict_make_plan(const mla_problem* problem, int32_t budget, int32_t sinks, int32_t recent,
                        mla_evict_plan* plan_out, size_t* workspace_bytes) {
  const int rc = check_cache_shape(problem);
  if (rc != MLA_OK) return rc;
  if (budget < 1 || sinks < 0 || recent < 0 || plan_out == nullptr) return MLA_ERR_INVALID_ARGUMENT;
  if (problem->batch > MLA_CHUNK_MAX_REQUESTS) return MLA_ERR_UNSUPPORTED;
  mla_evict_plan pl;
  std::memset(&pl, 0, sizeof(pl));
  pl.problem = *problem;
  pl.budget = budget;
  pl.sinks = sinks;
  pl.recent = recent;
  // a move fills a slot below the budget from one behind it
  const int64_t slots = static_cast<int64_t>(problem->max_pages_per_seq) * problem->page_size;
  const int64_t behind = slots > budget ? slots - budget : 0;
  pl.most_moves = behind < budget ? behind : budget;
  pl.ws_counts = 0;
  pl.ws_moves = align_up(static_cast<int64_t>(problem->batch) * 4);
  pl.workspace_bytes = align_up(pl.ws_moves + problem->batch * pl.most_moves * 8);
  pl.mark = kEvictPlanMark;
  *plan_out = pl;
  if (workspace_bytes) *workspace_bytes = static_cast<size_t>(pl.workspace_bytes);
  return MLA_OK;
}

int mla_cache_evict(const mla_evict_plan* plan, void* kv_cache, const int32_t* block_table,
                    const int32_t* seq_lens, const float* weights, const int32_t* positions,
                    int64_t stride, void* workspace, size_t workspace_bytes, int32_t* seq_lens_out,
                    float* weights_out, int32_t* positions_out, uint32_t* status,
                    mla_stream_t stream) {
  if (plan == nullptr || plan->mark != kEvictPlanMark) return MLA_ERR_INVALID_ARGUMENT;
  const mla_problem& pr = plan->problem;
  const int rc = check_cache_shape(&pr);
  if (rc != MLA_OK) return rc;
  if (!kv_cache || !block_table || !seq_lens || !weights || !positions || !workspace || !seq_lens_out ||
      !weights_out || !positions_out || stride < 1 || stride > INT64_MAX / 8 / (static_cast<int64_t>(pr.batch) + 1))
    return MLA_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < static_cast<size_t>(plan->workspace_bytes)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(kv_cache, 16) || !aligned(workspace, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(weights, 4) || !aligned(positions, 4) || !aligned(seq_lens_out, 4) || !aligned(weights_out, 4) ||
      !aligned(positions_out, 4) || !aligned(status, 4))
    return MLA_ERR_MISALIGNED;
  if (pr.batch == 0) return MLA_OK;
  const int64_t slots = entry_bytes(pr, stride);
  const Array written[] = {{kv_cache, cache_bytes(pr), nullptr}, {workspace, plan->workspace_bytes, nullptr},
                           {seq_lens_out, pr.batch * 4ll, seq_lens}, {weights_out, slots, weights},
                           {positions_out, slots, positions}, {status, 4, nullptr}};
  const Array read[] = {{block_table, table_bytes(pr), nullptr}, {seq_lens, pr.batch * 4ll, nullptr},
                        {weights, slots, nullptr}, {positions, slots, nullptr}};
  if (!stand_alone(written, read)) return MLA_ERR_INVALID_ARGUMENT;
  EvictParams p;
  p.kv = static_cast<uint8_t*>(kv_cache);
  p.block_table = block_table;
  p.lens = seq_lens;
  p.weights = weights;
  p.positions = positions;
  p.lens_out = seq_lens_out;
  p.weights_out = weights_out;
  p.positions_out = positions_out;
  p.counts = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + plan->ws_counts);
  p.moves = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + plan->ws_moves);
  p.status = status;
  p.stride = stride;
  p.most_moves = plan->most_moves;
  p.batch = pr.batch;
  p.budget = plan->budget;
  p.sinks = plan->sinks;
  p.recent = plan->recent;
  p.page_shift = shift_of(pr.page_size);
  p.num_pages = pr.num_pages;
  p.max_pages = pr.max_pages_per_seq;
  p.row_bytes = static_cast<int32_t>(row_bytes(pr.kv_dtype));
  return launch_cache_evict(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
