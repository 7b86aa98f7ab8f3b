// RMS norm of rows, with the residual's addition and 8-bit outputs:
// h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight.
//
// One pass over memory: a row stays in its threads' registers (in 32 bits)
// between the sum of its squares and its output, so x, the residual and the
// weight are read once and each output written once; that traffic is the
// bound.  Rows that consist of whole 16-byte pieces on 16-byte boundaries are
// owned by G threads, each with R pieces, piece i of thread t being number i *
// G + t of the row, so a warp's accesses are contiguous.  Other rows go in
// 32-bit words instead (mla_norm_words_kernel).
#include <cuda_runtime.h>

#include <type_traits>

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

// e4m3 codes of two values, the first in the low byte: nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(hi), "f"(lo));
  return two;
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

template <typename T, int kOut, int R, int G, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) mla_norm_kernel(const NormParams p) {
  __shared__ float slots[2][32];
  constexpr int V = 16 / sizeof(T);
  const int width = G == 0 ? blockDim.x : G;     // threads of a row
  const int t = G == 0 ? threadIdx.x : threadIdx.x % (G == 0 ? 1 : G);
  const int64_t row = G == 0 ? static_cast<int64_t>(blockIdx.x)
                             : static_cast<int64_t>(blockIdx.x) * (kRowThreads / (G == 0 ? 1 : G)) +
                                   threadIdx.x / (G == 0 ? 1 : G);
  // a group past the last row stays for its warp's shuffles
  const int pieces = G == 0 || row < p.rows ? p.cols / V : 0;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  const T* r = static_cast<const T*>(p.residual) + row * p.residual_stride;
  const T* w = static_cast<const T*>(p.weight);
  constexpr bool kWeightFirst = R * V < 32;   // else its registers are not to be had
  auto load = [&](const T* base, int i) {
    const int k = i * width + t;
    return k < pieces ? reinterpret_cast<const uint4*>(base)[k] : make_uint4(0, 0, 0, 0);
  };
  auto store = [&](T* base, int i, const float* v) {
    const int k = i * width + t;
    if (k < pieces) reinterpret_cast<uint4*>(base)[k] = pack16<T>(v);
  };
  after_predecessor();
  uint4 xe[R], re[R], we[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    xe[i] = load(x, i);
    if (p.residual) re[i] = load(r, i);
  }
  auto load_weight = [&] {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (p.weight) we[i] = load(w, i);
  };
  if (kWeightFirst) load_weight();
  float h[R * V];   // 0 where there is no piece
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float* v = h + i * V;
    unpack16<T>(xe[i], v);
    if (p.residual) {
      float b[V];
      unpack16<T>(re[i], b);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] += b[j];
    }
#pragma unroll
    for (int j = 0; j < V; ++j) sum = fmaf(v[j], v[j], sum);
  }
  if (p.residual_out) {
    T* ro = static_cast<T*>(p.residual_out) + row * p.residual_out_stride;
#pragma unroll
    for (int i = 0; i < R; ++i) store(ro, i, h + i * V);
  }
  if (!kWeightFirst) load_weight();
  const float rstd = rsqrtf(row_reduce<G, false>(sum, slots[0]) / static_cast<float>(p.cols) + p.eps);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float* v = h + i * V;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] *= rstd;
    if (p.weight) {
      float b[V];
      unpack16<T>(we[i], b);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] *= b[j];
    }
    if (kOut == MLA_NORM_OUT_E4M3_ROW) {
      const bool in = i * width + t < pieces;   // else 0 * inf is possible
#pragma unroll
      for (int j = 0; j < V; ++j) amax = max_nan(amax, in ? fabsf(v[j]) : 0.f);
    }
  }
  if (kOut == MLA_NORM_OUT_SAME) {
    T* out = static_cast<T*>(p.out) + row * p.out_stride;
#pragma unroll
    for (int i = 0; i < R; ++i) store(out, i, h + i * V);
    return;
  }
  uint8_t* out = static_cast<uint8_t*>(p.out) + row * p.out_stride;
  float inv = 1.f;
  if (kOut == MLA_NORM_OUT_E4M3_ROW) {
    const float scale = max_nan(row_reduce<G, true>(amax, slots[1]) / 448.f, kMinRowScale);
    inv = 1.f / scale;
    if (pieces && t == 0) static_cast<float*>(p.scales)[row] = scale;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int k = i * width + t;
    const float* v = h + i * V;
    bool any = true;
    if (kOut == MLA_NORM_OUT_E4M3_E8M0) {
      // a group of 32 is 32 / V neighbouring lanes' pieces
      float a = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) a = fmaxf(a, fabsf(v[j]));
#pragma unroll
      for (int o = 16 / V; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      any = a > 0.f;
      const uint32_t byte = e4m3_scale_byte(a);
      inv = scale_byte_reciprocal(byte);
      if (k < pieces && k % (32 / V) == 0)
        static_cast<uint8_t*>(p.scales)[row * p.scale_stride + k / (32 / V)] = static_cast<uint8_t>(byte);
    }
    uint32_t c[V / 4];
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      const float* y = v + 4 * j;
      c[j] = e4m3x2(y[0] * inv, y[1] * inv) | e4m3x2(y[2] * inv, y[3] * inv) << 16;
      if (!any) c[j] &= 0x7F7F7F7Fu;   // zeros without their signs (or NaN)
    }
    if (k < pieces && V == 8) reinterpret_cast<uint2*>(out)[k] = make_uint2(c[0], c[V / 4 - 1]);
    if (k < pieces && V == 4) reinterpret_cast<uint32_t*>(out)[k] = c[0];
  }
}

// Rows of any width at any element's address: 32-bit words of E elements,
// word i of a lane being number (warp * R + i) * 32 + lane of the row, so that
// each access of a warp is 128 contiguous bytes.  Where a row of 16-bit
// elements starts inside a word, a lane's word is put together from the two
// aligned ones around it (they hold at least one element of the row each, so
// the reads stay on the tensor's own words) and leaves in the aligned word
// that begins with the lane below's second element; the ends of a warp's words
// go as single elements.  All but the row's last words take the short paths
// without a comparison per element.
template <typename T, int kOut, int R, int G, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) mla_norm_words_kernel(const NormParams p) {
  __shared__ float slots[2][32];
  constexpr int E = Word<T>::kElems;
  using Half = typename std::conditional<E == 2, uint16_t, uint32_t>::type;   // an element's bits
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = G == 0 ? static_cast<int64_t>(blockIdx.x)
                             : static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + warp;
  const int k0 = (G == 0 ? warp * R * 32 : 0) + lane;
  // elements from the warp's first word, and from the lane's, to the row's end
  const int warp_left = (G == 0 || row < p.rows ? p.cols : 0) - (k0 - lane) * E, left = warp_left - lane * E;
  auto whole = [&](int i) { return warp_left >= 32 * E * (i + 1); };     // every lane's word i
  auto any = [&](int i) { return warp_left > 32 * E * i; };              // some lane's
  auto has = [&](int i, int elems) { return left >= 32 * E * i + elems; };
  auto load = [&](const void* base, int64_t stride, uint32_t (&w)[R]) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(static_cast<const T*>(base) + row * stride + k0 * E);
    const uint32_t* words = reinterpret_cast<const uint32_t*>(at & ~static_cast<uintptr_t>(3));
    const bool odd = E == 2 && (at & 2);
#pragma unroll
    for (int i = 0; i < R; ++i) w[i] = whole(i) || has(i, 1) ? words[32 * i] : 0u;
    if (odd) {
      uint32_t hi[R];
#pragma unroll
      for (int i = 0; i < R; ++i) hi[i] = whole(i) || has(i, 2) ? words[32 * i + 1] : 0u;
#pragma unroll
      for (int i = 0; i < R; ++i) w[i] = __funnelshift_r(w[i], hi[i], 16);
    } else if (E == 2) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (!whole(i) && !has(i, 2)) w[i] &= 0xFFFFu;
    }
  };
  auto store = [&](void* base, int64_t stride, const uint32_t (&w)[R]) {
    T* dst = static_cast<T*>(base) + row * stride + k0 * E;
    uint32_t* words = reinterpret_cast<uint32_t*>(reinterpret_cast<uintptr_t>(dst) & ~static_cast<uintptr_t>(3));
    Half* elem = reinterpret_cast<Half*>(dst);
    if (E == 1 || !(reinterpret_cast<uintptr_t>(dst) & 2)) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (whole(i) || has(i, E))
          words[32 * i] = w[i];
        else if (has(i, 1))
          elem[32 * E * i] = static_cast<Half>(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (!any(i)) continue;
        const uint32_t below = __shfl_up_sync(0xffffffffu, w[i], 1);
        if (lane > 0 ? has(i, 1) : false) words[32 * i] = __funnelshift_r(below, w[i], 16);
        if (lane == 0) elem[32 * E * i] = static_cast<Half>(w[i]);
        if (whole(i) ? lane == 31 : has(i, 2) && (lane == 31 || !has(i, 3)))
          elem[32 * E * i + 1] = static_cast<Half>(w[i] >> 16);
      }
    }
  };
  after_predecessor();
  uint32_t xw[R], rw[R];
  load(p.x, p.x_stride, xw);
  if (p.residual) load(p.residual, p.residual_stride, rw);
  float h[R * E];   // 0 where there is no element
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float* v = h + i * E;
    Word<T>::get(xw[i], v);
    if (p.residual) {
      float b[E];
      Word<T>::get(rw[i], b);
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] += b[j];
    }
#pragma unroll
    for (int j = 0; j < E; ++j) sum = fmaf(v[j], v[j], sum);
  }
  if (p.residual_out) {
#pragma unroll
    for (int i = 0; i < R; ++i) xw[i] = Word<T>::put(h + i * E);
    store(p.residual_out, p.residual_out_stride, xw);
  }
  if (p.weight) load(p.weight, 0, rw);
  const float rstd = rsqrtf(row_reduce<G, false>(sum, slots[0]) / static_cast<float>(p.cols) + p.eps);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float* v = h + i * E;
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] *= rstd;
    if (p.weight) {
      float b[E];
      Word<T>::get(rw[i], b);
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] *= b[j];
    }
    if (kOut != MLA_NORM_OUT_SAME && !whole(i)) {   // 0 where there is none: not 0 * inf
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (!has(i, j + 1)) v[j] = 0.f;
    }
    if (kOut == MLA_NORM_OUT_E4M3_ROW) {
#pragma unroll
      for (int j = 0; j < E; ++j) amax = max_nan(amax, fabsf(v[j]));
    }
  }
  if (kOut == MLA_NORM_OUT_SAME) {
#pragma unroll
    for (int i = 0; i < R; ++i) xw[i] = Word<T>::put(h + i * E);
    store(p.out, p.out_stride, xw);
    return;
  }
  float inv = 1.f;
  if (kOut == MLA_NORM_OUT_E4M3_ROW) {
    const float scale = max_nan(row_reduce<G, true>(amax, slots[1]) / 448.f, kMinRowScale);
    inv = 1.f / scale;
    if (has(0, 1) && k0 == 0) static_cast<float*>(p.scales)[row] = scale;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float* v = h + i * E;
    if (!any(i)) continue;
    bool some = true;
    if (kOut == MLA_NORM_OUT_E4M3_E8M0) {
      // a group of 32 is 32 / E neighbouring lanes' words
      float a = 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j) a = fmaxf(a, fabsf(v[j]));
#pragma unroll
      for (int o = 16 / E; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      some = a > 0.f;
      const uint32_t byte = e4m3_scale_byte(a);
      inv = scale_byte_reciprocal(byte);
      if (has(i, 1) && lane % (32 / E) == 0)
        static_cast<uint8_t*>(p.scales)[row * p.scale_stride + (k0 + 32 * i) * E / 32] = static_cast<uint8_t>(byte);
    }
    xw[i] = e4m3x2(v[0] * inv, v[E - 1] * inv);
    if (!some) xw[i] &= 0x7F7Fu;   // zeros without their signs (or NaN)
  }
  uint8_t* out = static_cast<uint8_t*>(p.out) + row * p.out_stride + k0 * E;
  if (E == 1) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (has(i, 1)) out[32 * i] = static_cast<uint8_t>(xw[i]);
  } else if (!(reinterpret_cast<uintptr_t>(out) & 1)) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (whole(i) || has(i, 2))
        reinterpret_cast<uint16_t*>(out)[32 * i] = static_cast<uint16_t>(xw[i]);
      else if (has(i, 1))
        out[64 * i] = static_cast<uint8_t>(xw[i]);
    }
  } else {   // as in store, by bytes
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (!any(i)) continue;
      const uint32_t below = __shfl_up_sync(0xffffffffu, xw[i], 1);
      if (lane > 0 ? has(i, 1) : false)
        reinterpret_cast<uint16_t*>(out - 1)[32 * i] = static_cast<uint16_t>((below >> 8) | (xw[i] << 8));
      if (lane == 0) out[64 * i] = static_cast<uint8_t>(xw[i]);
      if (whole(i) ? lane == 31 : has(i, 2) && (lane == 31 || !has(i, 3)))
        out[64 * i + 1] = static_cast<uint8_t>(xw[i] >> 8);
    }
  }
}

template <typename T, int kOut, bool kWords, int R, int G>
cudaError_t launch_one(const NormParams& p, int threads, cudaStream_t stream) {
  constexpr int kRows = G == 0 ? 1 : kRowThreads / (G == 0 ? 1 : G);
  const int blocks = p.rows / kRows + (p.rows % kRows != 0);
  auto launch = [&](auto kernel, int t) { return launch_dependent(kernel, blocks, t, stream, p); };
  if constexpr (kWords && G != 0)
    return launch(mla_norm_words_kernel<T, kOut, R, G, kRowThreads>, kRowThreads);
  else if constexpr (G != 0)
    return launch(mla_norm_kernel<T, kOut, R, G, kRowThreads>, kRowThreads);
  else if constexpr (kWords)
    return threads <= 256 ? launch(mla_norm_words_kernel<T, kOut, R, 0, 256>, threads)
                          : launch(mla_norm_words_kernel<T, kOut, R, 0, 1024>, threads);
  else
    return threads <= 256 ? launch(mla_norm_kernel<T, kOut, R, 0, 256>, threads)
                          : launch(mla_norm_kernel<T, kOut, R, 0, 1024>, threads);
}

template <typename T, int kOut>
cudaError_t launch_formed(const NormParams& p, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  constexpr int kOutBytes = kOut == MLA_NORM_OUT_SAME ? 16 : V;
  auto fits = [&](const void* base, int64_t stride, int bytes, int size) {
    return base == nullptr || (reinterpret_cast<uintptr_t>(base) % bytes == 0 &&
                               (p.rows == 1 || stride * size % bytes == 0));
  };
  const bool whole = p.cols % V == 0 && fits(p.x, p.x_stride, 16, sizeof(T)) &&
                     fits(p.residual, p.residual_stride, 16, sizeof(T)) && fits(p.weight, 0, 16, sizeof(T)) &&
                     fits(p.residual_out, p.residual_out_stride, 16, sizeof(T)) &&
                     fits(p.out, p.out_stride, kOutBytes, kOut == MLA_NORM_OUT_SAME ? sizeof(T) : 1);
  const bool many = p.rows >= 512;   // enough rows to fill the multiprocessors with few threads each
  auto threads = [](int units, int R) { return ((units + R - 1) / R + 31) / 32 * 32; };
  if (whole) {
    constexpr int kMost = sizeof(T) == 4 ? 8 : 4;   // pieces of a thread in a block of 1,024: the widest row
    const int n = p.cols / V;
    if (n <= 8) return launch_one<T, kOut, false, 1, 8>(p, 0, stream);
    if (n <= 32) return launch_one<T, kOut, false, 1, 32>(p, 0, stream);
    if (n <= 128 && many) return launch_one<T, kOut, false, 4, 32>(p, 0, stream);
    if (n <= 1024 && !many) return launch_one<T, kOut, false, 1, 0>(p, threads(n, 1), stream);
    if (n <= 4096) return launch_one<T, kOut, false, 4, 0>(p, threads(n, 4), stream);
    return launch_one<T, kOut, false, kMost, 0>(p, threads(n, kMost), stream);
  }
  constexpr int kMost = sizeof(T) == 4 ? 32 : 16;   // words of a thread
  const int n = (p.cols + Word<T>::kElems - 1) / Word<T>::kElems;
  if (n <= 128) return launch_one<T, kOut, true, 4, 32>(p, 0, stream);
  if (n <= 4096 && !many) return launch_one<T, kOut, true, 4, 0>(p, threads(n, 4), stream);
  if (n <= 16384) return launch_one<T, kOut, true, 16, 0>(p, threads(n, 16), stream);
  return launch_one<T, kOut, true, kMost, 0>(p, threads(n, kMost), stream);
}

template <typename T>
cudaError_t launch_typed(const NormParams& p, cudaStream_t stream) {
  if (p.out_format == MLA_NORM_OUT_SAME) return launch_formed<T, MLA_NORM_OUT_SAME>(p, stream);
  if (p.out_format == MLA_NORM_OUT_E4M3_E8M0) return launch_formed<T, MLA_NORM_OUT_E4M3_E8M0>(p, stream);
  return launch_formed<T, MLA_NORM_OUT_E4M3_ROW>(p, stream);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  if (p.dtype == MLA_DTYPE_BF16) return launch_typed<__nv_bfloat16>(p, stream);
  if (p.dtype == MLA_DTYPE_F16) return launch_typed<__half>(p, stream);
  return launch_typed<float>(p, stream);
}

}  // namespace mla
