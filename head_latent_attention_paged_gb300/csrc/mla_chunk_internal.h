// Internal declarations of the operators in include/mla_chunk.h.
#pragma once

#include "../../include/mla_chunk.h"
#include "mla_layer_internal.h"

namespace mla {

// What the attention and the weights read alike.
struct ChunkParams {
  const uint16_t* q;            // bf16 [tokens][heads][576]
  const int32_t* starts;        // [batch + 1]
  const uint8_t* kv;
  const int32_t* block_table;   // [batch][max_pages]
  const int32_t* lens;          // [batch]
  uint32_t* status;             // or null
  int32_t tokens, batch, heads;
  int32_t page_shift, num_pages, max_pages, kv_dtype, causal;
  float scale_log2;             // sm_scale * log2(e)
};

struct AttendParams {
  ChunkParams c;
  uint16_t* o;                  // bf16 [tokens][heads][512]
  float* lse;                   // [tokens][heads]
};
struct WeightsParams {
  ChunkParams c;
  const float* lse;
  const float* in;              // [batch][stride], or null
  float* out;                   // [batch][stride]
  int64_t stride;
};

struct ChunkWorkspace {
  float* part_o;                // [2 * clusters][64][128][8]
  float* part_lse;              // [2 * clusters][128]
  int32_t* segments;            // [2 * clusters][4]
  int2* starts;                 // [batch + 1] each request's first expanded row, and how many of its
                                // rows there is room for; null: rows are read in pages
  uint16_t* rows;               // bf16 [capacity][576]
  int32_t context, capacity;    // rows of requests there is room for, and with each one's padding
  int32_t clusters;
};
constexpr int kDensePad = 32;   // an expanded request's rows end with zeros to a multiple of this
cudaError_t launch_chunk_attend(const AttendParams& p, const ChunkWorkspace& w, cudaStream_t stream);

cudaError_t launch_cache_weights(const WeightsParams& p, const ChunkWorkspace& w, cudaStream_t stream);

// A quantised cache's rows, of the requests that have new tokens, as bf16 rows
// one request behind the other, each with its padding.
cudaError_t launch_expand(const ChunkParams& p, const ChunkWorkspace& w, cudaStream_t stream);

constexpr int kMaxChunkClusters = 512;   // of a plan: more SMs are taken as 1,024
constexpr int kSmemAttrChunk = 16, kSmemAttrWeights = 17, kSmemAttrEvict = 18;   // slots of set_smem_attr_once

struct EvictParams {
  uint8_t* kv;
  const int32_t* block_table;
  const int32_t* lens;
  const float* weights;
  const int32_t* positions;
  int32_t* lens_out;
  float* weights_out;
  int32_t* positions_out;
  int32_t* counts;              // [batch] rows to move
  int32_t* moves;               // [batch][most_moves][2]: slot to, slot from
  uint32_t* status;             // or null
  int64_t stride, most_moves;
  int32_t batch, budget, sinks, recent;
  int32_t page_shift, num_pages, max_pages, row_bytes;
};
cudaError_t launch_cache_evict(const EvictParams& p, cudaStream_t stream);

#ifdef __CUDACC__
// A request's new tokens and cached rows; what lies outside its bounds is
// taken as the nearest one (`bad` says so).
struct ChunkRequest {
  int32_t first, count, len;
  bool bad;
  ChunkRequest() = default;
  __device__ __forceinline__ ChunkRequest(const ChunkParams& p, int32_t b) {
    const int32_t s = p.starts[b], e = p.starts[b + 1], l = p.lens[b];
    const int32_t most = p.max_pages << p.page_shift;
    first = min(max(s, 0), p.tokens);
    count = min(max(e, first), p.tokens) - first;
    len = min(max(l, 0), most);
    bad = s != first || e != first + count || l != len;
  }
  __device__ __forceinline__ ChunkRequest(int32_t rows, int32_t tokens) : first(0), count(tokens), len(rows), bad(false) {}
  // rows that token j of the request sees
  __device__ __forceinline__ int32_t seen(int32_t j, int32_t causal) const {
    return causal ? min(max(len - count + j + 1, 0), len) : len;
  }
};
#endif

}  // namespace mla
