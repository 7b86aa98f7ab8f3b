// Host side of include/mla_layer.h: argument checks, the rotary table and the
// launches.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "mla_layer_internal.h"

using namespace mla;

namespace {

constexpr int32_t kRopePlanMark = 0x524F5031;   // set by mla_rope_make_plan

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

int dtype_size(int32_t dtype) {
  return dtype == MLA_DTYPE_BF16 || dtype == MLA_DTYPE_F16 ? 2 : dtype == MLA_DTYPE_F32 ? 4 : 0;
}

// A set of equally spaced rows in memory, in bytes.
struct Rows {
  const void* base;
  int64_t stride, width, count;
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(base); }
  uintptr_t end() const { return begin() + static_cast<uintptr_t>((count - 1) * stride + width); }
  bool same(const Rows& o) const { return base == o.base && (stride == o.stride || count == 1); }
};

// Whether two sets of rows share memory.  Columns of one buffer (equal
// strides, as the slices of a fused projection) are told apart; other
// interleavings count as shared.
bool overlap(const Rows& a, const Rows& b) {
  if (a.base == nullptr || b.base == nullptr || a.end() <= b.begin() || b.end() <= a.begin()) return false;
  if (a.count < 2 || b.count < 2 || a.stride != b.stride) return true;
  const uintptr_t s = static_cast<uintptr_t>(a.stride);
  const uintptr_t d = b.begin() >= a.begin() ? (b.begin() - a.begin()) % s : (s - (a.begin() - b.begin()) % s) % s;
  return d < static_cast<uintptr_t>(a.width) || d + static_cast<uintptr_t>(b.width) > s;
}

bool span_fits(int64_t count, int64_t stride, int64_t size) {   // (count - 1) * stride * size in 62 bits
  return count < 2 || stride <= (INT64_MAX / 2) / size / (count - 1);
}

int check_rope_config(const mla_rope_config& c) {
  if ((c.layout != MLA_ROPE_INTERLEAVED && c.layout != MLA_ROPE_HALVES) || c.rope_dim < 2 ||
      c.rope_dim > MLA_ROPE_MAX_DIM || c.rope_dim % 2 != 0 || c.scaling < MLA_ROPE_SCALING_NONE ||
      c.scaling > MLA_ROPE_SCALING_YARN)
    return MLA_ERR_UNSUPPORTED;
  if (!std::isfinite(c.theta) || c.theta <= 1.0 || !std::isfinite(c.amplitude) || c.amplitude < 0.0)
    return MLA_ERR_INVALID_ARGUMENT;
  if (c.scaling != MLA_ROPE_SCALING_NONE && (!std::isfinite(c.factor) || c.factor <= 0.0))
    return MLA_ERR_INVALID_ARGUMENT;
  if ((c.scaling == MLA_ROPE_SCALING_PARTS || c.scaling == MLA_ROPE_SCALING_YARN) &&
      (c.original_positions < 1 || !std::isfinite(c.fast_rotations) || !(c.slow_rotations > 0.0) ||
       !(c.fast_rotations > c.slow_rotations)))
    return MLA_ERR_INVALID_ARGUMENT;
  return MLA_OK;
}

int check_rope_plan(const mla_rope_plan* plan) {
  if (plan == nullptr || plan->reserved != kRopePlanMark) return MLA_ERR_INVALID_ARGUMENT;
  return check_rope_config(plan->config);
}

template <int kPairs>
void fill_table(const mla_rope_plan& plan, RopeTable<kPairs>* t) {
  const int pairs = plan.config.rope_dim / 2;
  std::memset(t, 0, sizeof(*t));
  for (int i = 0; i < pairs && i < kPairs; ++i) t->turns[i] = plan.turns[i];
  t->amplitude = plan.amplitude;
  t->halves = plan.config.layout == MLA_ROPE_HALVES;
}

// What the append and the gather check alike.
int fill_tokens(const mla_problem* pr, int32_t tokens, const int32_t* positions,
                const int32_t* requests, const int32_t* block_table, const void* kv,
                const void* dense, int64_t dense_stride, uint32_t* status, TokenParams* t) {
  const int rc = check_cache_shape(pr);
  if (rc != MLA_OK) return rc;
  if (tokens < 0 || dense_stride < kDqk || !span_fits(tokens, dense_stride, 2)) return MLA_ERR_INVALID_ARGUMENT;
  if (dense_stride % 8 != 0) return MLA_ERR_MISALIGNED;
  if (tokens == 0) return MLA_OK;
  if (!positions || !block_table || !kv || !dense) return MLA_ERR_INVALID_ARGUMENT;
  if (requests == nullptr && (pr->batch < 1 || tokens % pr->batch != 0)) return MLA_ERR_INVALID_ARGUMENT;
  if (!aligned(dense, 16) || !aligned(kv, 16) || !aligned(positions, 4) || !aligned(requests, 4) ||
      !aligned(block_table, 4) || !aligned(status, 4))
    return MLA_ERR_MISALIGNED;
  t->positions = positions;
  t->requests = requests;
  t->block_table = block_table;
  t->status = status;
  t->tokens = tokens;
  t->per_request = requests ? 1 : tokens / pr->batch;
  t->batch = pr->batch;
  t->page_shift = pr->page_size == 16 ? 4 : pr->page_size == 32 ? 5 : pr->page_size == 64 ? 6 : 7;
  t->num_pages = pr->num_pages;
  t->max_pages = pr->max_pages_per_seq;
  t->kv_dtype = pr->kv_dtype;
  return MLA_OK;
}

int64_t cache_bytes(const mla_problem& pr) {
  const int64_t row = pr.kv_dtype == MLA_KV_BF16 ? kDqk * 2 : pr.kv_dtype == MLA_KV_FP8_E4M3_E8M0 ? kFp8RowBytes : kFp4RowBytes;
  return static_cast<int64_t>(pr.num_pages) * pr.page_size * row;
}

}  // namespace

extern "C" {

int mla_rms_norm(const mla_norm_problem* problem, const void* x, const void* residual,
                 const void* weight, void* residual_out, void* out, void* scales,
                 mla_stream_t stream) {
  if (problem == nullptr) return MLA_ERR_INVALID_ARGUMENT;
  const mla_norm_problem& pr = *problem;
  const int size = dtype_size(pr.dtype);
  if (size == 0 || pr.out_format < MLA_NORM_OUT_SAME || pr.out_format > MLA_NORM_OUT_E4M3_ROW ||
      pr.cols > MLA_NORM_MAX_COLS)
    return MLA_ERR_UNSUPPORTED;
  const bool mx = pr.out_format == MLA_NORM_OUT_E4M3_E8M0;
  const int out_size = pr.out_format == MLA_NORM_OUT_SAME ? size : 1;
  const int64_t groups = (pr.cols + 31) / 32;
  if (pr.rows < 0 || pr.cols < 1 || !std::isfinite(pr.eps) || pr.eps < 0.f || pr.reserved != 0 ||
      pr.x_stride < pr.cols || pr.out_stride < pr.cols || (mx && pr.scale_stride < groups) ||
      (residual && pr.residual_stride < pr.cols) ||
      (residual_out && (!residual || pr.residual_out_stride < pr.cols)) ||
      !span_fits(pr.rows, pr.x_stride, size) || !span_fits(pr.rows, pr.out_stride, out_size) ||
      (mx && !span_fits(pr.rows, pr.scale_stride, 1)) ||
      (residual && !span_fits(pr.rows, pr.residual_stride, size)) ||
      (residual_out && !span_fits(pr.rows, pr.residual_out_stride, size)))
    return MLA_ERR_INVALID_ARGUMENT;
  if (pr.rows == 0) return MLA_OK;
  if (!x || !out || (scales != nullptr) != (pr.out_format != MLA_NORM_OUT_SAME)) return MLA_ERR_INVALID_ARGUMENT;
  if (!aligned(x, size) || !aligned(residual, size) || !aligned(weight, size) ||
      !aligned(residual_out, size) || !aligned(out, out_size) || (!mx && !aligned(scales, 4)))
    return MLA_ERR_MISALIGNED;
  const Rows rx{x, pr.x_stride * size, static_cast<int64_t>(pr.cols) * size, pr.rows};
  const Rows rr{residual, pr.residual_stride * size, static_cast<int64_t>(pr.cols) * size, pr.rows};
  const Rows rw{weight, 0, static_cast<int64_t>(pr.cols) * size, 1};
  const Rows ro{residual_out, pr.residual_out_stride * size, static_cast<int64_t>(pr.cols) * size, pr.rows};
  const Rows ry{out, pr.out_stride * out_size, static_cast<int64_t>(pr.cols) * out_size, pr.rows};
  const Rows rs{scales, mx ? pr.scale_stride : 4, mx ? groups : 4, pr.rows};
  const bool typed = pr.out_format == MLA_NORM_OUT_SAME;   // may stand on an input's elements
  if (overlap(ry, ro) || overlap(rs, ry) || overlap(rs, ro) || overlap(rs, rx) || overlap(rs, rr) ||
      overlap(rs, rw) || overlap(ry, rw) || overlap(ro, rw) ||
      (overlap(ry, rx) && !(typed && ry.same(rx))) || (overlap(ry, rr) && !(typed && ry.same(rr))) ||
      (overlap(ro, rx) && !ro.same(rx)) || (overlap(ro, rr) && !ro.same(rr)))
    return MLA_ERR_INVALID_ARGUMENT;
  NormParams p;
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.residual_out = residual_out;
  p.out = out;
  p.scales = scales;
  p.x_stride = pr.x_stride;
  p.residual_stride = pr.residual_stride;
  p.residual_out_stride = pr.residual_out_stride;
  p.out_stride = pr.out_stride;
  p.scale_stride = pr.scale_stride;
  p.rows = pr.rows;
  p.cols = pr.cols;
  p.dtype = pr.dtype;
  p.out_format = pr.out_format;
  p.eps = pr.eps;
  p.inv_cols = 1.f / static_cast<float>(pr.cols);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = pr.dtype == MLA_DTYPE_BF16  ? launch_norm_of<__nv_bfloat16>(p, st)
                          : pr.dtype == MLA_DTYPE_F16 ? launch_norm_of<__half>(p, st)
                                                      : launch_norm_of<float>(p, st);
  return err == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_rope_make_plan(const mla_rope_config* config, mla_rope_plan* plan_out) {
  if (config == nullptr || plan_out == nullptr) return MLA_ERR_INVALID_ARGUMENT;
  const mla_rope_config c = *config;
  const int rc = check_rope_config(c);
  if (rc != MLA_OK) return rc;
  const double two_pi = 6.283185307179586476925286766559;
  const double log_theta = std::log(c.theta);
  const int pairs = c.rope_dim / 2;
  double low = 0.0, high = 0.0;
  if (c.scaling == MLA_ROPE_SCALING_YARN) {
    auto pair_of = [&](double rotations) {
      return c.rope_dim * std::log(c.original_positions / (rotations * two_pi)) / (2.0 * log_theta);
    };
    low = std::fmax(std::floor(pair_of(c.fast_rotations)), 0.0);
    high = std::fmin(std::ceil(pair_of(c.slow_rotations)), c.rope_dim - 1.0);
  }
  mla_rope_plan plan;
  std::memset(&plan, 0, sizeof(plan));
  plan.config = c;
  for (int i = 0; i < pairs; ++i) {
    const double f = std::pow(c.theta, -2.0 * i / c.rope_dim);
    double w = 1.0;   // share of the unscaled frequency
    if (c.scaling == MLA_ROPE_SCALING_LINEAR) {
      w = 0.0;
    } else if (c.scaling == MLA_ROPE_SCALING_PARTS) {
      const double t = c.original_positions * f / two_pi;
      w = std::fmin(std::fmax((t - c.slow_rotations) / (c.fast_rotations - c.slow_rotations), 0.0), 1.0);
    } else if (c.scaling == MLA_ROPE_SCALING_YARN) {
      w = 1.0 - std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
    }
    const double g = c.scaling == MLA_ROPE_SCALING_NONE ? f : w * f + (1.0 - w) * (f / c.factor);
    if (!std::isfinite(g)) return MLA_ERR_INVALID_ARGUMENT;
    // the fraction of a turn per position in 2^-64ths: whole turns do not count
    const double turns = g / two_pi;
    const double scaled = std::ldexp(turns - std::floor(turns), 64);
    plan.turns[i] = scaled >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(scaled);
  }
  const double own = c.scaling == MLA_ROPE_SCALING_YARN && c.factor > 1.0 ? 0.1 * std::log(c.factor) + 1.0 : 1.0;
  plan.amplitude = static_cast<float>(c.amplitude > 0.0 ? c.amplitude : own);
  if (!std::isfinite(plan.amplitude) || plan.amplitude <= 0.f) return MLA_ERR_INVALID_ARGUMENT;
  plan.reserved = kRopePlanMark;
  *plan_out = plan;
  return MLA_OK;
}

int mla_rope(const mla_rope_problem* problem, const mla_rope_plan* plan, const void* x,
             const int32_t* positions, void* out, mla_stream_t stream) {
  if (problem == nullptr) return MLA_ERR_INVALID_ARGUMENT;
  const mla_rope_problem& pr = *problem;
  int rc = check_rope_plan(plan);
  if (rc != MLA_OK) return rc;
  const int size = dtype_size(pr.dtype);
  if (size == 0) return MLA_ERR_UNSUPPORTED;
  const int64_t T = pr.tokens, H = pr.num_heads, D = pr.head_dim;
  if (T < 0 || H < 1 || D < 1 || pr.rope_offset < 0 || pr.rope_offset > D - plan->config.rope_dim ||
      (pr.transposed != 0 && pr.transposed != 1) || pr.x_token_stride < 0 || pr.x_head_stride < 0 ||
      pr.out_token_stride < 0 || pr.out_head_stride < 0 || !span_fits(T, pr.x_token_stride, size) ||
      !span_fits(H, pr.x_head_stride, size) || !span_fits(T, pr.out_token_stride, size) ||
      !span_fits(H, pr.out_head_stride, size))
    return MLA_ERR_INVALID_ARGUMENT;
  if (H * D > INT32_MAX / 64 || pr.x_token_stride > INT32_MAX || pr.x_head_stride > INT32_MAX ||
      pr.out_token_stride > INT32_MAX || pr.out_head_stride > INT32_MAX)
    return MLA_ERR_UNSUPPORTED;
  if (T == 0) return MLA_OK;
  const int64_t out_heads = (H - 1) * pr.out_head_stride, out_tokens = (T - 1) * pr.out_token_stride;
  const int64_t x_heads = (H - 1) * pr.x_head_stride, x_tokens = (T - 1) * pr.x_token_stride;
  // distinct elements of out: heads within a token's stride, or tokens within a head's
  const bool token_major = (H == 1 || pr.out_head_stride >= D) && (T == 1 || pr.out_token_stride >= out_heads + D);
  const bool head_major = (T == 1 || pr.out_token_stride >= D) && (H == 1 || pr.out_head_stride >= out_tokens + D);
  if (!token_major && !head_major) return MLA_ERR_INVALID_ARGUMENT;
  if (!x || !positions || !out) return MLA_ERR_INVALID_ARGUMENT;
  if (!aligned(x, size) || !aligned(out, size) || !aligned(positions, 4)) return MLA_ERR_MISALIGNED;
  const bool in_place = x == out && (T == 1 || pr.x_token_stride == pr.out_token_stride) &&
                        (H == 1 || pr.x_head_stride == pr.out_head_stride);
  // tokens as rows, each over all its heads, and heads as rows, each over all
  // its tokens: x and out are apart where either of the two are
  const Rows xt{x, pr.x_token_stride * size, (x_heads + D) * size, T}, ot{out, pr.out_token_stride * size, (out_heads + D) * size, T};
  const Rows xh{x, pr.x_head_stride * size, (x_tokens + D) * size, H}, oh{out, pr.out_head_stride * size, (out_tokens + D) * size, H};
  const Rows rp{positions, 0, T * 4, 1};
  if ((!in_place && overlap(xt, ot) && overlap(xh, oh)) || overlap(ot, rp)) return MLA_ERR_INVALID_ARGUMENT;
  RopeParams p;
  p.x = x;
  p.out = out;
  p.positions = positions;
  p.x_token_stride = static_cast<int32_t>(pr.x_token_stride);
  p.x_head_stride = static_cast<int32_t>(pr.x_head_stride);
  p.out_token_stride = static_cast<int32_t>(pr.out_token_stride);
  p.out_head_stride = static_cast<int32_t>(pr.out_head_stride);
  p.tokens = pr.tokens;
  p.heads = pr.num_heads;
  p.head_dim = pr.head_dim;
  p.offset = pr.rope_offset;
  p.dim = plan->config.rope_dim;
  p.dtype = pr.dtype;
  p.transposed = pr.transposed;
  fill_table(*plan, &p.table);
  return launch_rope(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_cache_append_tokens(const mla_problem* problem, int32_t tokens, const void* rows,
                            int64_t row_stride, const int32_t* positions, const int32_t* requests,
                            const int32_t* block_table, const void* norm_weight, float norm_eps,
                            const mla_rope_plan* rope, void* kv_cache, uint32_t* status,
                            mla_stream_t stream) {
  AppendTokensParams p;
  int rc = fill_tokens(problem, tokens, positions, requests, block_table, kv_cache, rows, row_stride, status, &p.t);
  if (rc != MLA_OK) return rc;
  if (norm_weight && (!std::isfinite(norm_eps) || norm_eps < 0.f)) return MLA_ERR_INVALID_ARGUMENT;
  if (!aligned(norm_weight, 16)) return MLA_ERR_MISALIGNED;
  if (rope) {
    rc = check_rope_plan(rope);
    if (rc != MLA_OK) return rc;
    if (rope->config.rope_dim != kDr) return MLA_ERR_UNSUPPORTED;
  }
  if (tokens == 0) return MLA_OK;
  const Rows rs{rows, row_stride * 2, kDqk * 2, tokens}, rk{kv_cache, 0, cache_bytes(*problem), 1};
  if (overlap(rs, rk)) return MLA_ERR_INVALID_ARGUMENT;
  p.rows = static_cast<const uint16_t*>(rows);
  p.row_stride = row_stride;
  p.weight = static_cast<const uint16_t*>(norm_weight);
  p.eps = norm_eps;
  p.kv = static_cast<uint8_t*>(kv_cache);
  p.rotate = rope != nullptr;
  if (rope)
    fill_table(*rope, &p.table);
  else
    std::memset(&p.table, 0, sizeof(p.table));
  return launch_append_tokens(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

int mla_cache_gather(const mla_problem* problem, int32_t tokens, const void* kv_cache,
                     const int32_t* positions, const int32_t* requests,
                     const int32_t* block_table, void* out, int64_t out_stride, uint32_t* status,
                     mla_stream_t stream) {
  GatherParams p;
  const int rc = fill_tokens(problem, tokens, positions, requests, block_table, kv_cache, out, out_stride, status, &p.t);
  if (rc != MLA_OK) return rc;
  if (tokens == 0) return MLA_OK;
  const Rows ro{out, out_stride * 2, kDqk * 2, tokens}, rk{kv_cache, 0, cache_bytes(*problem), 1};
  if (overlap(ro, rk)) return MLA_ERR_INVALID_ARGUMENT;
  p.kv = static_cast<const uint8_t*>(kv_cache);
  p.out = static_cast<uint16_t*>(out);
  p.out_stride = out_stride;
  return launch_gather(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
