// RMS norm of rows, with the residual's addition and 8-bit outputs:
// h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight.
//
// One pass over memory: a row stays in its threads' registers (in 32 bits)
// between the sum of its squares and its output, so x, the residual and the
// weight are read once and each output written once; that traffic is the
// bound.  A group of G threads owns a row, each with R pieces of kVec
// elements (16 bytes where the rows allow it, single elements otherwise), piece
// i of thread t being number i * G + t of the row, so a warp's accesses are
// contiguous.
#include <cuda_runtime.h>

#include "mla_layer_internal.h"
#include "mla_quant.cuh"
#include "mla_types.cuh"

namespace mla {

namespace {

constexpr float kMinRowScale = 1.17549435e-38f;   // 2^-126
constexpr int kRowThreads = 128;                  // block size where a warp or less owns a row

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int G, bool kMax>
__device__ __forceinline__ float lanes_reduce(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? max_nan(v, w) : v + w;
  }
  return v;
}

// Over the row's threads: G lanes of a warp, or (G = 0) the whole block
// through one slot of shared memory per warp.
template <int G, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* slots) {
  if (G != 0) return lanes_reduce<G == 0 ? 32 : G, kMax>(v);
  v = lanes_reduce<32, kMax>(v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) slots[warp] = v;
  __syncthreads();
  v = lane < (blockDim.x >> 5) ? slots[lane] : 0.f;   // sums and maxima of magnitudes start at 0
  return lanes_reduce<32, kMax>(v);
}

template <int kBytes>
struct Piece;
template <>
struct Piece<16> { using type = uint4; };
template <>
struct Piece<8> { using type = uint2; };
template <>
struct Piece<4> { using type = uint32_t; };
template <>
struct Piece<2> { using type = uint16_t; };
template <>
struct Piece<1> { using type = uint8_t; };

// kVec elements as one access.
template <typename T, int kVec>
union Elems {
  typename Piece<sizeof(T) * kVec>::type raw;
  T v[kVec];
  __device__ Elems() {}
};

template <typename T, int kOut, int kVec, int R, int G, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) mla_norm_kernel(const NormParams p) {
  __shared__ float slots[2][32];
  const int width = G == 0 ? blockDim.x : G;     // threads of a row
  const int t = G == 0 ? threadIdx.x : threadIdx.x % (G == 0 ? 1 : G);
  const int64_t row = G == 0 ? static_cast<int64_t>(blockIdx.x)
                             : static_cast<int64_t>(blockIdx.x) * (kRowThreads / (G == 0 ? 1 : G)) +
                                   threadIdx.x / (G == 0 ? 1 : G);
  const int pieces = p.cols / kVec;              // kVec divides cols
  // a group past the last row stays for its warp's shuffles
  const bool live = G == 0 || row < p.rows;
  using E = Elems<T, kVec>;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  const T* r = static_cast<const T*>(p.residual) + row * p.residual_stride;
  const T* w = static_cast<const T*>(p.weight);
  constexpr bool kWeightFirst = R * kVec < 32;   // else its registers are not to be had
  E xe[R], re[R], we[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int k = i * width + t;
    if (live && k < pieces) {
      xe[i].raw = reinterpret_cast<const decltype(E::raw)*>(x)[k];
      if (p.residual) re[i].raw = reinterpret_cast<const decltype(E::raw)*>(r)[k];
    }
  }
  auto load_weight = [&] {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int k = i * width + t;
      if (p.weight && live && k < pieces) we[i].raw = reinterpret_cast<const decltype(E::raw)*>(w)[k];
    }
  };
  if (kWeightFirst) load_weight();
  float h[R * kVec];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const bool in = live && i * width + t < pieces;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      float v = in ? to_f32(xe[i].v[j]) : 0.f;
      if (in && p.residual) v += to_f32(re[i].v[j]);
      h[i * kVec + j] = v;
      sum = fmaf(v, v, sum);
    }
  }
  if (p.residual_out) {
    T* ro = static_cast<T*>(p.residual_out) + row * p.residual_out_stride;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int k = i * width + t;
      E e;
#pragma unroll
      for (int j = 0; j < kVec; ++j) e.v[j] = from_f32<T>(h[i * kVec + j]);
      if (live && k < pieces) reinterpret_cast<decltype(E::raw)*>(ro)[k] = e.raw;
    }
  }
  if (!kWeightFirst) load_weight();
  const float rstd = rsqrtf(row_reduce<G, false>(sum, slots[0]) / static_cast<float>(p.cols) + p.eps);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const bool in = live && i * width + t < pieces;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      float y = h[i * kVec + j] * rstd;
      if (p.weight) y = in ? y * to_f32(we[i].v[j]) : 0.f;
      if (kOut != MLA_NORM_OUT_SAME && !in) y = 0.f;   // 0 * inf of an unused piece
      h[i * kVec + j] = y;
      if (kOut == MLA_NORM_OUT_E4M3_ROW) amax = max_nan(amax, fabsf(y));
    }
  }
  if (kOut == MLA_NORM_OUT_SAME) {
    T* out = static_cast<T*>(p.out) + row * p.out_stride;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int k = i * width + t;
      E e;
#pragma unroll
      for (int j = 0; j < kVec; ++j) e.v[j] = from_f32<T>(h[i * kVec + j]);
      if (live && k < pieces) reinterpret_cast<decltype(E::raw)*>(out)[k] = e.raw;
    }
    return;
  }
  uint8_t* out = static_cast<uint8_t*>(p.out) + row * p.out_stride;
  float inv = 1.f;
  if (kOut == MLA_NORM_OUT_E4M3_ROW) {
    const float scale = max_nan(row_reduce<G, true>(amax, slots[1]) / 448.f, kMinRowScale);
    inv = 1.f / scale;
    if (live && t == 0) static_cast<float*>(p.scales)[row] = scale;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int k = i * width + t;
    bool any = true;
    if (kOut == MLA_NORM_OUT_E4M3_E8M0) {
      // a group of 32 is 32 / kVec neighbouring lanes' pieces
      float a = 0.f;
#pragma unroll
      for (int j = 0; j < kVec; ++j) a = fmaxf(a, fabsf(h[i * kVec + j]));
#pragma unroll
      for (int o = 16 / kVec; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      any = a > 0.f;
      const int e = any ? max(-127, min(127, ceil_log2_over_448(a))) : -127;
      inv = pow2_neg(e);
      if (live && k < pieces && k % (32 / kVec) == 0)
        static_cast<uint8_t*>(p.scales)[row * p.scale_stride + k / (32 / kVec)] = static_cast<uint8_t>(e + 127);
    }
    Elems<uint8_t, kVec> c;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const float y = h[i * kVec + j];
      c.v[j] = static_cast<uint8_t>(any || y != y ? f32_to_e4m3(y * inv) : 0u);
    }
    if (live && k < pieces) reinterpret_cast<decltype(c.raw)*>(out)[k] = c.raw;
  }
}

template <typename T, int kOut, int kVec, int R, int G>
void launch_one(const NormParams& p, int threads, cudaStream_t stream) {
  constexpr int kRows = G == 0 ? 1 : kRowThreads / (G == 0 ? 1 : G);
  const int blocks = p.rows / kRows + (p.rows % kRows != 0);
  if constexpr (G != 0)
    mla_norm_kernel<T, kOut, kVec, R, G, kRowThreads><<<blocks, kRowThreads, 0, stream>>>(p);
  else if (threads <= 256)
    mla_norm_kernel<T, kOut, kVec, R, 0, 256><<<blocks, threads, 0, stream>>>(p);
  else
    mla_norm_kernel<T, kOut, kVec, R, 0, 1024><<<blocks, threads, 0, stream>>>(p);
}

template <typename T, int kOut>
void launch_formed(const NormParams& p, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  constexpr int kOutBytes = kOut == MLA_NORM_OUT_SAME ? 16 : V;
  auto fits = [&](const void* base, int64_t stride, int bytes, int size) {
    return base == nullptr || (reinterpret_cast<uintptr_t>(base) % bytes == 0 && stride * size % bytes == 0);
  };
  const bool vec = p.cols % V == 0 && fits(p.x, p.x_stride, 16, sizeof(T)) &&
                   fits(p.residual, p.residual_stride, 16, sizeof(T)) && fits(p.weight, 0, 16, sizeof(T)) &&
                   fits(p.residual_out, p.residual_out_stride, 16, sizeof(T)) &&
                   fits(p.out, p.out_stride, kOutBytes, kOut == MLA_NORM_OUT_SAME ? sizeof(T) : 1);
  const int pieces = vec ? p.cols / V : p.cols;
  auto threads = [&](int R) { return ((pieces + R - 1) / R + 31) / 32 * 32; };
  if (vec) {
    if (pieces <= 8) return launch_one<T, kOut, V, 1, 8>(p, 0, stream);
    if (pieces <= 32) return launch_one<T, kOut, V, 1, 32>(p, 0, stream);
    if (pieces <= 128 && p.rows >= 512) return launch_one<T, kOut, V, 4, 32>(p, 0, stream);
    if (pieces <= 1024 && p.rows < 512) return launch_one<T, kOut, V, 1, 0>(p, threads(1), stream);
    if (pieces <= 4096) return launch_one<T, kOut, V, 4, 0>(p, threads(4), stream);
    return launch_one<T, kOut, V, 32 / V, 0>(p, threads(32 / V), stream);
  }
  if (pieces <= 128) return launch_one<T, kOut, 1, 4, 32>(p, 0, stream);
  if (pieces <= 8192) return launch_one<T, kOut, 1, 8, 0>(p, threads(8), stream);
  return launch_one<T, kOut, 1, 32, 0>(p, threads(32), stream);
}

template <typename T>
void launch_typed(const NormParams& p, cudaStream_t stream) {
  if (p.out_format == MLA_NORM_OUT_SAME)
    launch_formed<T, MLA_NORM_OUT_SAME>(p, stream);
  else if (p.out_format == MLA_NORM_OUT_E4M3_E8M0)
    launch_formed<T, MLA_NORM_OUT_E4M3_E8M0>(p, stream);
  else
    launch_formed<T, MLA_NORM_OUT_E4M3_ROW>(p, stream);
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
