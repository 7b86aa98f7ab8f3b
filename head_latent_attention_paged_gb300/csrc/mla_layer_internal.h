// Internal declarations of the operators in include/mla_layer.h.
#pragma once

#include "../../include/mla_layer.h"
#include "mla_internal.h"

namespace mla {

// The layer operators are launched as programmatic dependents of whatever
// precedes them on their stream: the launch itself, and the set-up before
// after_predecessor(), overlap the predecessor's tail.  A kernel touches no
// memory but its parameters before that call, after which everything the
// predecessor wrote is visible; it then lets its own successor start, which
// waits in the same way until this kernel has completed.  (Small calls one
// after another: 4.1 -> 1.4 us each.)
#ifdef __CUDACC__
__device__ __forceinline__ void after_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 blocks, int threads, int smem,
                             cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = blocks;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

struct NormParams {
  const void* x;
  const void* residual;         // or null
  const void* weight;           // or null
  void* residual_out;           // or null
  void* out;
  void* scales;
  int64_t x_stride, residual_stride, residual_out_stride, out_stride, scale_stride;
  int32_t rows, cols;
  int32_t dtype, out_format;
  float eps, inv_cols;          // inv_cols: 1 / cols
};
// For the element types of MLA_DTYPE_*, each in a source of its own.
template <typename T>
cudaError_t launch_norm_of(const NormParams& p, cudaStream_t stream);

// A rotation as the kernels take it, by value: pair i turns by turns[i] *
// pos (wrapping) 2^-64ths of a turn.
template <int kPairs>
struct RopeTable {
  uint64_t turns[kPairs];
  float amplitude;
  int32_t halves;               // layout: 1 = MLA_ROPE_HALVES
};

struct RopeParams {
  const void* x;
  void* out;
  const int32_t* positions;
  int32_t x_token_stride, x_head_stride, out_token_stride, out_head_stride;
  int32_t tokens, heads, head_dim, offset, dim;
  int32_t dtype, transposed;
  RopeTable<MLA_ROPE_MAX_DIM / 2> table;
};
cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream);

struct TokenParams {            // the append's and the gather's common part
  const int32_t* positions;
  const int32_t* requests;      // or null: token t is request t / per_request
  const int32_t* block_table;
  uint32_t* status;             // or null
  int32_t tokens, per_request;
  int32_t batch, page_shift, num_pages, max_pages;   // pages of 2^page_shift tokens
  int32_t kv_dtype;
};

struct AppendTokensParams {
  TokenParams t;
  const uint16_t* rows;
  int64_t row_stride;
  const uint16_t* weight;       // or null
  float eps;
  uint8_t* kv;
  int32_t rotate;               // 1: table is valid
  RopeTable<kDr / 2> table;
};
cudaError_t launch_append_tokens(const AppendTokensParams& p, cudaStream_t stream);

struct GatherParams {
  TokenParams t;
  const uint8_t* kv;
  uint16_t* out;
  int64_t out_stride;
};
cudaError_t launch_gather(const GatherParams& p, cudaStream_t stream);

}  // namespace mla
