// Rotary positions on part of each head.
#include <cuda_runtime.h>

#include "mla_layer_internal.h"
#include "mla_turn.cuh"
#include "mla_types.cuh"

namespace mla {

namespace {

constexpr int kRopeThreads = 256;

// One block per token: the token's cosines and sines once into shared memory,
// then every element of its heads.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) mla_rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs[MLA_ROPE_MAX_DIM / 2];
  const int64_t t = blockIdx.x;
  const int32_t pos = p.positions[t];
  if (pos < 0) return;
  const int pairs = p.dim >> 1;
  for (int i = threadIdx.x; i < pairs; i += kRopeThreads) {
    float c, s;
    turn_cos_sin(p.table.turns[i], pos, &c, &s);
    cs[i] = make_float2(c * p.table.amplitude, (p.transposed ? -s : s) * p.table.amplitude);
  }
  __syncthreads();
  const T* x = static_cast<const T*>(p.x) + t * p.x_token_stride;
  T* out = static_cast<T*>(p.out) + t * p.out_token_stride;
  for (int64_t k = threadIdx.x; k < static_cast<int64_t>(p.heads) * pairs; k += kRopeThreads) {
    const int64_t head = k / pairs;
    const int i = static_cast<int>(k - head * pairs);
    const int a = p.offset + (p.table.halves ? i : 2 * i), b = a + (p.table.halves ? pairs : 1);
    const T* xh = x + head * p.x_head_stride;
    T* oh = out + head * p.out_head_stride;
    const float va = to_f32(xh[a]), vb = to_f32(xh[b]);
    oh[a] = from_f32<T>(va * cs[i].x - vb * cs[i].y);
    oh[b] = from_f32<T>(va * cs[i].y + vb * cs[i].x);
  }
  const int rest = p.head_dim - p.dim;
  if (p.x == p.out || rest == 0) return;
  for (int64_t k = threadIdx.x; k < static_cast<int64_t>(p.heads) * rest; k += kRopeThreads) {
    const int64_t head = k / rest;
    const int i = static_cast<int>(k - head * rest);
    const int e = i < p.offset ? i : i + p.dim;
    out[head * p.out_head_stride + e] = x[head * p.x_head_stride + e];
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  if (p.tokens == 0) return cudaSuccess;
  if (p.dtype == MLA_DTYPE_BF16)
    mla_rope_kernel<__nv_bfloat16><<<p.tokens, kRopeThreads, 0, stream>>>(p);
  else if (p.dtype == MLA_DTYPE_F16)
    mla_rope_kernel<__half><<<p.tokens, kRopeThreads, 0, stream>>>(p);
  else
    mla_rope_kernel<float><<<p.tokens, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
