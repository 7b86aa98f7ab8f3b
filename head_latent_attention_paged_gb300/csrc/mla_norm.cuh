// RMS norm of rows, with the residual's addition and 8-bit outputs (compiled once
// for each element type, mla_norm_*.cu):
// h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight.
//
// One pass over memory: a row stays in its threads' registers (in 32 bits)
// between the sum of its squares and its output, so x, the residual and the
// weight are read once and each output written once; that traffic is the
// bound.  Rows that consist of whole 16-byte pieces on 16-byte boundaries are
// owned by G threads, each with R pieces, piece i of thread t being number i *
// G + t of the row, so a warp's accesses are contiguous (mla_norm_kernel).
// Other rows go in 32-bit words instead (mla_norm_words_kernel).
#pragma once

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

// 1 / sqrt(v) with one Newton step whose residual 1 - v r^2 is formed exactly
// (the product and its rounding error), so that the result is off by little
// more than its own rounding.
__device__ __forceinline__ float rsqrt_exact(float v) {
  const float r = rsqrtf(v);
  const float p = v * r, p_low = fmaf(v, r, -p);
  const float rest = fmaf(-p_low, r, fmaf(-p, r, 1.f));
  const float better = fmaf(0.5f * r, rest, r);
  return fabsf(rest) < 1.f ? better : r;   // zero, infinite and NaN v keep theirs
}

// h * rstd * w; where it decides a group's power of two, with the first
// product's rounding error taken along, since a scale on the other side of its
// border halves or doubles all its codes.
template <int kOut>
__device__ __forceinline__ float norm_product(float h, float rstd, float w) {
  const float p = h * rstd;
  // p + 0: the error of a product that is -0 has to be -0 as well, or their sum
  // is +0
  return kOut == MLA_NORM_OUT_E4M3_E8M0 ? fmaf(p, w, fmaf(h, rstd, -(p + 0.f)) * w) : p * w;
}

// The scale of a row, amax / 448 to nearest (tried for every mantissa), at least
// 2^-126, and NaN or infinite with amax.
__device__ __forceinline__ float row_scale(float amax) {
  const float q = amax * (1.f / 448.f);
  const float s = fmaf(-fmaf(q, 448.f, -amax), 1.f / 448.f, q);
  return max_nan(amax == INFINITY ? amax : s, kMinRowScale);
}

// y / scale to nearest, from -y and neg_inv, -1 / scale to nearest: the product
// and its remainder's share.  (By the negatives a zero keeps its sign, and two
// values go through packed arithmetic.)  scale is 0 in the place of an infinite
// one, whose quotients are 0.
__device__ __forceinline__ float2 quotients(float2 neg_y, float scale, float neg_inv) {
  const float2 inv = make_float2(neg_inv, neg_inv);
  const float2 q = __fmul2_rn(neg_y, inv);
  return __ffma2_rn(__ffma2_rn(q, make_float2(scale, scale), neg_y), inv, q);
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

// 1 / sqrt(mean(h^2) + eps) of a row from its threads' sums of squares.  Where
// the squares leave the range of 32 bits (a mean below 2^-100, whose small terms
// were lost, or past the largest number) h is scaled by a power of two and they
// are summed again: small rows by 2^100, which is exact, large ones by 2^-34, by
// which no value loses bits whose product is not lost as well (a row's mean is
// past 2^112, so a product of 2^-149 comes from 2^-93), and by 2^-38 more for
// their squares alone.  Infinite values keep their infinite sum.  The squares
// of f16 values do not get that far.  One step after another, by their
// volatile order, since registers for more would be taken from every row.
template <typename T, int G, int N>
__device__ __forceinline__ float row_rstd(float (&h)[N], float sum, const NormParams& p, float (*slots)[32]) {
  const float mean = row_reduce<G, false>(sum, slots[0]) * p.inv_cols + p.eps;
  if (std::is_same<T, __half>::value) return rsqrt_exact(mean);
  const bool small = mean < 0x1p-100f, large = mean == INFINITY;
  // one decision for all threads that reduce together
  if (G == 0 || G == 32 ? small || large : __any_sync(0xffffffffu, small || large)) {
    const float f = small ? 0x1p100f : large ? 0x1p-34f : 1.f, g = large ? 0x1p-38f : 1.f;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      asm volatile("{\n .reg .f32 v;\n mul.f32 %0, %0, %2;\n mul.f32 v, %0, %3;\n fma.rn.f32 %1, v, v, %1;\n}"
                   : "+f"(h[i]), "+f"(sum)
                   : "f"(f), "f"(g));
    return rsqrt_exact(row_reduce<G, false>(sum, slots[1]) * p.inv_cols + p.eps * f * g * f * g) * g;
  }
  return rsqrt_exact(mean);
}

// Rows of whole 16-byte pieces.  Bound by memory: 16384 x 4096 bf16 with a
// residual to e4m3 with group scales 69.6 us, 6.78 TB/s, 1.00 of the measured
// copy rate; with row scales 69.0; 8192 x 4096 bf16 with a residual to bf16 40.1
// us, 0.99.
template <typename T, int kOut, int R, int G, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, 1024 / kMaxThreads)   // at most 64 registers
    mla_norm_kernel(const NormParams p) {
  __shared__ float slots[3][32];
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
  constexpr float kSign = kOut == MLA_NORM_OUT_E4M3_ROW ? -1.f : 1.f;   // for quotients()
  const float rstd = kSign * row_rstd<T, G>(h, sum, p, slots);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float* v = h + i * V;
    if (p.weight) {
      float b[V];
      unpack16<T>(we[i], b);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = norm_product<kOut>(v[j], rstd, b[j]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] *= rstd;
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
  float inv = 1.f, scale = 1.f;
  if (kOut == MLA_NORM_OUT_E4M3_ROW) {
    scale = row_scale(row_reduce<G, true>(amax, slots[2]));
    inv = -1.f / scale;
    if (pieces && t == 0) static_cast<float*>(p.scales)[row] = scale;
    if (scale == INFINITY) scale = 0.f;
  }
  auto codes = [&](float a, float b) {
    const float2 y = kOut == MLA_NORM_OUT_E4M3_ROW ? quotients(make_float2(a, b), scale, inv) : make_float2(a * inv, b * inv);
    return e4m3x2(y.x, y.y);
  };
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
      c[j] = codes(y[0], y[1]) | codes(y[2], y[3]) << 16;
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
// go as single elements.  A warp whose words the row has all of (kAll) goes
// without a comparison for each.  5003 x 2881 f16 with a residual to e4m3 with
// row scales: 25.4 us, 4.0 TB/s.  Neither memory nor the issue slots are full (a
// warp runs 72 instructions for 32 words, issued in 60 % of the cycles): at 64
// registers 28 warps fit a multiprocessor, and they wait for their loads, for one
// another at the row's two sums and for shuffles.  Left after measuring them for
// that case: 16-byte pieces shifted between lanes 41.7 us, the row staged through
// shared memory around its 16-byte lines 28.1 us.
template <typename T, int kOut, int R, int G, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) mla_norm_words_kernel(const NormParams p) {
  __shared__ float slots[3][32];
  constexpr int E = Word<T>::kElems;
  using Half = typename std::conditional<E == 2, uint16_t, uint32_t>::type;   // an element's bits
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = G == 0 ? static_cast<int64_t>(blockIdx.x)
                             : static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + warp;
  const int k0 = (G == 0 ? warp * R * 32 : 0) + lane;
  // elements from the lane's first word to the row's end
  const int left = (G == 0 || row < p.rows ? p.cols : 0) - k0 * E;
  const bool all = left + lane * E >= 32 * E * R;   // of the warp: the same for its lanes
  using All = std::true_type;
  using Some = std::false_type;
  // whether word i has so many elements
  auto has = [&](auto kAll, int i, int elems) { return decltype(kAll)::value || left >= 32 * E * i + elems; };
  // whether its last element is stored by its own lane: no lane behind it has one
  auto last = [&](auto kAll, int i) {
    return decltype(kAll)::value ? lane == 31 : has(kAll, i, 2) && (lane == 31 || !has(kAll, i, 3));
  };
  auto load_as = [&](auto kAll, uintptr_t at, uint32_t (&w)[R]) {
    const uint32_t* words = reinterpret_cast<const uint32_t*>(at & ~static_cast<uintptr_t>(3));
#pragma unroll
    for (int i = 0; i < R; ++i) w[i] = has(kAll, i, 1) ? words[32 * i] : 0u;
    if (E == 2 && (at & 2)) {
      uint32_t hi[R];
#pragma unroll
      for (int i = 0; i < R; ++i) hi[i] = has(kAll, i, 2) ? words[32 * i + 1] : 0u;
#pragma unroll
      for (int i = 0; i < R; ++i) w[i] = __funnelshift_r(w[i], hi[i], 16);
    } else if (E == 2) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (!has(kAll, i, 2)) w[i] &= 0xFFFFu;
    }
  };
  auto load = [&](const void* base, int64_t stride, uint32_t (&w)[R]) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(static_cast<const T*>(base) + row * stride + k0 * E);
    if (all)
      load_as(All(), at, w);
    else
      load_as(Some(), at, w);
  };
  auto store_as = [&](auto kAll, T* dst, const uint32_t (&w)[R]) {
    uint32_t* words = reinterpret_cast<uint32_t*>(reinterpret_cast<uintptr_t>(dst) & ~static_cast<uintptr_t>(3));
    Half* elem = reinterpret_cast<Half*>(dst);
    if (E == 1 || !(reinterpret_cast<uintptr_t>(dst) & 2)) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (has(kAll, i, E))
          words[32 * i] = w[i];
        else if (has(kAll, i, 1))
          elem[32 * E * i] = static_cast<Half>(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint32_t below = __shfl_up_sync(0xffffffffu, w[i], 1);
        if (lane > 0 && has(kAll, i, 1)) words[32 * i] = __funnelshift_r(below, w[i], 16);
        if (lane == 0 && has(kAll, i, 1)) elem[32 * E * i] = static_cast<Half>(w[i]);
        if (last(kAll, i)) elem[32 * E * i + 1] = static_cast<Half>(w[i] >> 16);
      }
    }
  };
  auto store = [&](void* base, int64_t stride, const uint32_t (&w)[R]) {
    T* dst = static_cast<T*>(base) + row * stride + k0 * E;
    if (all)
      store_as(All(), dst, w);
    else
      store_as(Some(), dst, w);
  };
  auto store_codes_as = [&](auto kAll, uint8_t* dst, const uint32_t (&c)[R]) {
    if (E == 1) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (has(kAll, i, 1)) dst[32 * i] = static_cast<uint8_t>(c[i]);
    } else if (!(reinterpret_cast<uintptr_t>(dst) & 1)) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (has(kAll, i, 2))
          reinterpret_cast<uint16_t*>(dst)[32 * i] = static_cast<uint16_t>(c[i]);
        else if (has(kAll, i, 1))
          dst[64 * i] = static_cast<uint8_t>(c[i]);
      }
    } else {   // as in store_as, by bytes
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint32_t below = __shfl_up_sync(0xffffffffu, c[i], 1);
        if (lane > 0 && has(kAll, i, 1))
          reinterpret_cast<uint16_t*>(dst - 1)[32 * i] = static_cast<uint16_t>((below >> 8) | (c[i] << 8));
        if (lane == 0 && has(kAll, i, 1)) dst[64 * i] = static_cast<uint8_t>(c[i]);
        if (last(kAll, i)) dst[64 * i + 1] = static_cast<uint8_t>(c[i] >> 8);
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
  constexpr float kSign = kOut == MLA_NORM_OUT_E4M3_ROW ? -1.f : 1.f;   // for quotients()
  const float rstd = kSign * row_rstd<T, G>(h, sum, p, slots);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float* v = h + i * E;
    if (p.weight) {
      float b[E];
      Word<T>::get(rw[i], b);
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = norm_product<kOut>(v[j], rstd, b[j]);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] *= rstd;
    }
  }
  if (kOut == MLA_NORM_OUT_SAME) {
#pragma unroll
    for (int i = 0; i < R; ++i) xw[i] = Word<T>::put(h + i * E);
    store(p.out, p.out_stride, xw);
    return;
  }
  if (!all) {   // 0 where there is none: not 0 * inf
#pragma unroll
    for (int i = 0; i < R * E; ++i)
      if (!has(Some(), i / E, i % E + 1)) h[i] = 0.f;
  }
  float inv = 1.f, scale = 1.f;
  if (kOut == MLA_NORM_OUT_E4M3_ROW) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < R * E; ++i) amax = max_nan(amax, fabsf(h[i]));
    scale = row_scale(row_reduce<G, true>(amax, slots[2]));
    inv = -1.f / scale;
    if (left > 0 && k0 == 0) static_cast<float*>(p.scales)[row] = scale;
    if (scale == INFINITY) scale = 0.f;
  }
  auto codes = [&](float a, float b) {
    const float2 y = kOut == MLA_NORM_OUT_E4M3_ROW ? quotients(make_float2(a, b), scale, inv) : make_float2(a * inv, b * inv);
    return e4m3x2(y.x, y.y);
  };
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float* v = h + i * E;
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
      if (lane % (32 / E) == 0 && has(Some(), i, 1))
        static_cast<uint8_t*>(p.scales)[row * p.scale_stride + (k0 + 32 * i) * E / 32] = static_cast<uint8_t>(byte);
    }
    xw[i] = codes(v[0], v[E - 1]);
    if (!some) xw[i] &= 0x7F7Fu;   // zeros without their signs (or NaN)
  }
  uint8_t* out = static_cast<uint8_t*>(p.out) + row * p.out_stride + k0 * E;
  if (all)
    store_codes_as(All(), out, xw);
  else
    store_codes_as(Some(), out, xw);
}

template <typename T, int kOut, bool kWords, int R, int G>
cudaError_t launch_one(const NormParams& p, int threads, cudaStream_t stream) {
  constexpr int kRows = G == 0 ? 1 : kRowThreads / (G == 0 ? 1 : G);
  const int blocks = p.rows / kRows + (p.rows % kRows != 0);
  auto launch = [&](auto kernel, int t) { return launch_dependent(kernel, blocks, t, 0, stream, p); };
  auto kernel = [](auto most) {   // most: the registers are shared out for that many threads
    if constexpr (kWords)
      return mla_norm_words_kernel<T, kOut, R, G, decltype(most)::value>;
    else
      return mla_norm_kernel<T, kOut, R, G, decltype(most)::value>;
  };
  if constexpr (G != 0) return launch(kernel(std::integral_constant<int, kRowThreads>()), kRowThreads);
  if (threads <= 256) return launch(kernel(std::integral_constant<int, 256>()), threads);
  return launch(kernel(std::integral_constant<int, 1024>()), threads);
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
  // Few rows: many threads for each, so that one row takes little time; many:
  // fewer threads with more pieces, since each joins the row's sums.  bf16 with
  // a residual to bf16, rows x cols, us with one piece a thread and with four: 64 x
  // 4096 1.9 and 2.1, 256 x 4096 2.3 and 2.5, 512 x 4096 3.0 and 3.1, 2048 x 8192
  // 23.4 and 21.6, 4096 x 4096 21.7 and 21.4.  Up to 128 pieces many rows have a
  // warp each: 512 x 512 1.8 (a block each: 2.1), 16384 x 512 12.0 (17.6), 16384 x
  // 1024 21.2 (21.6), up to 32 pieces half a warp: 16384 x 128 3.3 (a warp: 5.0), and
  // up to 8 pieces 8 lanes: 16384 x 64 2.4 (5.0).
  const bool many = p.rows >= 512;
  auto threads = [](int units, int R) { return ((units + R - 1) / R + 31) / 32 * 32; };
  if (whole) {
    constexpr int kMost = sizeof(T) == 4 ? 8 : 4;   // pieces of a thread in a block of 1,024: the widest row
    const int n = p.cols / V;
    if (n <= 8) return launch_one<T, kOut, false, 1, 8>(p, 0, stream);
    if (n <= 32 && many) return launch_one<T, kOut, false, 2, 16>(p, 0, stream);
    if (n <= 32) return launch_one<T, kOut, false, 1, 32>(p, 0, stream);
    if (n <= 128 && many) return launch_one<T, kOut, false, 4, 32>(p, 0, stream);
    if (n <= 1024 && !many) return launch_one<T, kOut, false, 1, 0>(p, threads(n, 1), stream);
    if (n <= 4096) return launch_one<T, kOut, false, 4, 0>(p, threads(n, 4), stream);
    return launch_one<T, kOut, false, kMost, 0>(p, threads(n, kMost), stream);
  }
  // Words of a thread, by the same rule: few rows 4 (128 x 2881 bf16 with a
  // residual 2.6 us, 8 words 3.2, 16 4.5).  Many rows 12 where that leaves no more
  // places empty than 8, else 8: 5003 x 2881 f16 with a residual to e4m3 with row
  // scales 4 28.6, 8 27.2, 12 25.5, 16 30.9 us, 3359 x 7466 f16 without one 8 27.9,
  // 12 22.8, but 16384 x 777 bf16 with one 8 25.1, 12 32.2.  Up to 256 and 384 words
  // many rows have a warp each: 14607 x 481 bf16 without a residual 7.6 us (a block
  // each: 15.5), 18503 x 708 f16 with one to e4m3 with group scales 27.5 (27.7, with
  // 8 words 32.6).  Wide rows 16, since 1,024 threads have 64 registers each: 4000 x
  // 8191 f32 with a residual to e4m3 with group scales 82 us (8 words: 89).
  constexpr int kMost = sizeof(T) == 4 ? 32 : 16;
  const int n = (p.cols + Word<T>::kElems - 1) / Word<T>::kElems;
  if (n <= 128) return launch_one<T, kOut, true, 4, 32>(p, 0, stream);
  if (n <= 256 && many) return launch_one<T, kOut, true, 8, 32>(p, 0, stream);
  if (n <= 2048 && !many) return launch_one<T, kOut, true, 4, 0>(p, threads(n, 4), stream);
  if (n <= 384 && many) return launch_one<T, kOut, true, 12, 32>(p, 0, stream);
  if (n <= 6144 && (n + 383) / 384 * 384 <= (n + 255) / 256 * 256)
    return launch_one<T, kOut, true, 12, 0>(p, threads(n, 12), stream);
  if (n <= 4096) return launch_one<T, kOut, true, 8, 0>(p, threads(n, 8), stream);
  if (n <= 16384) return launch_one<T, kOut, true, 16, 0>(p, threads(n, 16), stream);
  return launch_one<T, kOut, true, kMost, 0>(p, threads(n, kMost), stream);
}

}  // namespace

template <typename T>
cudaError_t launch_norm_of(const NormParams& p, cudaStream_t stream) {
  if (p.out_format == MLA_NORM_OUT_SAME) return launch_formed<T, MLA_NORM_OUT_SAME>(p, stream);
  if (p.out_format == MLA_NORM_OUT_E4M3_E8M0) return launch_formed<T, MLA_NORM_OUT_E4M3_E8M0>(p, stream);
  return launch_formed<T, MLA_NORM_OUT_E4M3_ROW>(p, stream);
}

}  // namespace mla
