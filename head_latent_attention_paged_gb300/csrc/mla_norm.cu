// RMS norm of rows, with the residual's addition and 8-bit outputs:
// h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight.
#include <cuda_runtime.h>

#include "mla_layer_internal.h"
#include "mla_quant.cuh"
#include "mla_types.cuh"

namespace mla {

namespace {

constexpr int kNormThreads = 256;
constexpr float kMinRowScale = 1.17549435e-38f;   // 2^-126

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <bool kMax>
__device__ __forceinline__ float block_reduce(float v, float* smem) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? max_nan(v, w) : v + w;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  __syncthreads();
  if (lane == 0) smem[warp] = v;
  __syncthreads();
  v = smem[0];
  for (int i = 1; i < warps; ++i) v = kMax ? max_nan(v, smem[i]) : v + smem[i];
  return v;
}

template <typename T, int kOut>
__global__ void __launch_bounds__(kNormThreads) mla_norm_kernel(const NormParams p) {
  __shared__ float smem[32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  const T* r = p.residual ? static_cast<const T*>(p.residual) + row * p.residual_stride : nullptr;
  const T* w = static_cast<const T*>(p.weight);
  T* ro = p.residual_out ? static_cast<T*>(p.residual_out) + row * p.residual_out_stride : nullptr;
  const int cols32 = (p.cols + 31) & ~31;   // whole warps, for the groups
  float sum = 0.f;
  for (int c = threadIdx.x; c < p.cols; c += kNormThreads) {
    const float v = to_f32(x[c]) + (r ? to_f32(r[c]) : 0.f);
    sum = fmaf(v, v, sum);
  }
  const float rstd = rsqrtf(block_reduce<false>(sum, smem) / p.cols + p.eps);
  auto value = [&](int c) {
    const float v = to_f32(x[c]) + (r ? to_f32(r[c]) : 0.f);
    return v * rstd * (w ? to_f32(w[c]) : 1.f);
  };
  float scale = 1.f, inv = 1.f;
  if (kOut == MLA_NORM_OUT_E4M3_ROW) {
    float amax = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += kNormThreads) amax = max_nan(amax, fabsf(value(c)));
    scale = max_nan(block_reduce<true>(amax, smem) / 448.f, kMinRowScale);
    inv = 1.f / scale;
    if (threadIdx.x == 0) static_cast<float*>(p.scales)[row] = scale;
  }
  for (int c = threadIdx.x; c < cols32; c += kNormThreads) {
    const bool in = c < p.cols;
    const float y = in ? value(c) : 0.f;
    const float hv = in ? to_f32(x[c]) + (r ? to_f32(r[c]) : 0.f) : 0.f;
    if (kOut == MLA_NORM_OUT_SAME) {
      if (in) (static_cast<T*>(p.out) + row * p.out_stride)[c] = from_f32<T>(y);
    } else if (kOut == MLA_NORM_OUT_E4M3_ROW) {
      if (in) (static_cast<uint8_t*>(p.out) + row * p.out_stride)[c] = static_cast<uint8_t>(f32_to_e4m3(y * inv));
    } else {
      float amax = fabsf(y);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = amax > 0.f ? max(-127, min(127, ceil_log2_over_448(amax))) : -127;
      if (in) {
        const uint32_t code = amax > 0.f || y != y ? f32_to_e4m3(y * pow2_neg(e)) : 0u;
        (static_cast<uint8_t*>(p.out) + row * p.out_stride)[c] = static_cast<uint8_t>(code);
        if ((c & 31) == 0)
          static_cast<uint8_t*>(p.scales)[row * p.scale_stride + (c >> 5)] = static_cast<uint8_t>(e + 127);
      }
    }
    if (in && ro) ro[c] = from_f32<T>(hv);
  }
}

template <typename T>
void launch_typed(const NormParams& p, cudaStream_t stream) {
  if (p.out_format == MLA_NORM_OUT_SAME)
    mla_norm_kernel<T, MLA_NORM_OUT_SAME><<<p.rows, kNormThreads, 0, stream>>>(p);
  else if (p.out_format == MLA_NORM_OUT_E4M3_E8M0)
    mla_norm_kernel<T, MLA_NORM_OUT_E4M3_E8M0><<<p.rows, kNormThreads, 0, stream>>>(p);
  else
    mla_norm_kernel<T, MLA_NORM_OUT_E4M3_ROW><<<p.rows, kNormThreads, 0, stream>>>(p);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  if (p.dtype == MLA_DTYPE_BF16)
    launch_typed<__nv_bfloat16>(p, stream);
  else if (p.dtype == MLA_DTYPE_F16)
    launch_typed<__half>(p, stream);
  else
    launch_typed<float>(p, stream);
  return cudaGetLastError();
}

}  // namespace mla
