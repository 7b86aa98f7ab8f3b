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
#include "sm103_ptx.cuh"

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
  return kOut == MLA_NORM_OUT_E4M3_E8M0 ? fmaf(p, w, fmaf(h, rstd, -p) * w) : p * w;
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
  const float rstd = rsqrt_exact(row_reduce<G, false>(sum, slots[0]) * p.inv_cols + p.eps);
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
  float inv = 1.f;
  if (kOut == MLA_NORM_OUT_E4M3_ROW) {
    const float scale = max_nan(row_reduce<G, true>(amax, slots[1]) * (1.f / 448.f), kMinRowScale);
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
// go as single elements.  Rows too wide to be staged, or too few.
template <typename T, int kOut, int R, int G, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) mla_norm_words_kernel(const NormParams p) {
  __shared__ float slots[2][32];
  constexpr int E = Word<T>::kElems;
  using Half = typename std::conditional<E == 2, uint16_t, uint32_t>::type;   // an element's bits
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = G == 0 ? static_cast<int64_t>(blockIdx.x)
                             : static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + warp;
  const int k0 = (G == 0 ? warp * R * 32 : 0) + lane;
  // elements from the lane's first word to the row's end
  const int left = (G == 0 || row < p.rows ? p.cols : 0) - k0 * E;
  auto has = [&](int i, int elems) { return left >= 32 * E * i + elems; };
  auto load = [&](const void* base, int64_t stride, uint32_t (&w)[R]) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(static_cast<const T*>(base) + row * stride + k0 * E);
    const uint32_t* words = reinterpret_cast<const uint32_t*>(at & ~static_cast<uintptr_t>(3));
    const bool odd = E == 2 && (at & 2);
#pragma unroll
    for (int i = 0; i < R; ++i) w[i] = has(i, 1) ? words[32 * i] : 0u;
    if (odd) {
      uint32_t hi[R];
#pragma unroll
      for (int i = 0; i < R; ++i) hi[i] = has(i, 2) ? words[32 * i + 1] : 0u;
#pragma unroll
      for (int i = 0; i < R; ++i) w[i] = __funnelshift_r(w[i], hi[i], 16);
    } else if (E == 2) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (!has(i, 2)) w[i] &= 0xFFFFu;
    }
  };
  auto store = [&](void* base, int64_t stride, const uint32_t (&w)[R]) {
    T* dst = static_cast<T*>(base) + row * stride + k0 * E;
    uint32_t* words = reinterpret_cast<uint32_t*>(reinterpret_cast<uintptr_t>(dst) & ~static_cast<uintptr_t>(3));
    Half* elem = reinterpret_cast<Half*>(dst);
    if (E == 1 || !(reinterpret_cast<uintptr_t>(dst) & 2)) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (has(i, E))
          words[32 * i] = w[i];
        else if (has(i, 1))
          elem[32 * E * i] = static_cast<Half>(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint32_t below = __shfl_up_sync(0xffffffffu, w[i], 1);
        if (lane > 0 && has(i, 1)) words[32 * i] = __funnelshift_r(below, w[i], 16);
        if (lane == 0 && has(i, 1)) elem[32 * E * i] = static_cast<Half>(w[i]);
        if (has(i, 2) && (lane == 31 || !has(i, 3)))
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
  const float rstd = rsqrt_exact(row_reduce<G, false>(sum, slots[0]) * p.inv_cols + p.eps);
  float amax = 0.f;
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
    if (kOut != MLA_NORM_OUT_SAME) {   // 0 where there is none: not 0 * inf
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
    const float scale = max_nan(row_reduce<G, true>(amax, slots[1]) * (1.f / 448.f), kMinRowScale);
    inv = 1.f / scale;
    if (has(0, 1) && k0 == 0) static_cast<float*>(p.scales)[row] = scale;
  }
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
      if (has(i, 2))
        reinterpret_cast<uint16_t*>(out)[32 * i] = static_cast<uint16_t>(xw[i]);
      else if (has(i, 1))
        out[64 * i] = static_cast<uint8_t>(xw[i]);
    }
  } else {   // as in store, by bytes
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const uint32_t below = __shfl_up_sync(0xffffffffu, xw[i], 1);
      if (lane > 0 && has(i, 1))
        reinterpret_cast<uint16_t*>(out - 1)[32 * i] = static_cast<uint16_t>((below >> 8) | (xw[i] << 8));
      if (lane == 0 && has(i, 1)) out[64 * i] = static_cast<uint8_t>(xw[i]);
      if (has(i, 2) && (lane == 31 || !has(i, 3)))
        out[64 * i + 1] = static_cast<uint8_t>(xw[i] >> 8);
    }
  }
}

// Many rows that the 16-byte pieces do not fit: a row passes through shared
// memory, where it lies as it does around its 16-byte boundaries, so that
// global memory sees 16-byte accesses (but for the row's ends) while the
// threads take words of E elements, word t + i * kWidth for thread t.  A block
// stays for several rows: the weights stay in registers, and the next
// row is copied in asynchronously while one is computed.
// Blocks of a multiprocessor, all resident at once, as far as registers go.
__host__ __device__ constexpr int staged_resident(int width, int words) {
  return width > 128 ? 2 : words > 12 ? 5 : 6;
}

__host__ __device__ inline int staged_buffer(int cols, int size) { return (cols * size + 15) / 16 * 16 + 16; }

// A row's place: its elements start `shift` bytes into 16-byte line 0; lines
// first .. end - 1 belong to it whole.
struct Lines {
  uint8_t* line;                 // global, 16-byte aligned
  int shift, first, end;
  __device__ __forceinline__ Lines(const void* row, int bytes) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row);
    shift = static_cast<int>(at & 15);
    line = reinterpret_cast<uint8_t*>(at - shift);
    first = (shift + 15) >> 4;
    end = (shift + bytes) >> 4;
  }
  // Byte offset of the element of the row's ends that lane l moves (0-15 those
  // in front of the whole lines, 16-31 those behind), or -1.  Rows have at
  // least one whole line.
  __device__ __forceinline__ int edge(int l, int size, int bytes) const {
    const int at = l < 16 ? shift + l * size : 16 * end + (l - 16) * size;
    return at < (l < 16 ? 16 * first : shift + bytes) ? at : -1;
  }
};

// R words of each thread between registers and a row in shared memory that
// starts on any element; words that the row does not have are skipped (n: the
// elements from the thread's first word to the row's end).
template <typename T, int kWidth, int R>
__device__ __forceinline__ void read_words(uint32_t (&w)[R], const uint8_t* row, int n) {
  constexpr int E = Word<T>::kElems;
  if (E == 1 || !(reinterpret_cast<uintptr_t>(row) & 2)) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < R; ++i) w[i] = n > E * kWidth * i ? p[kWidth * i] : 0u;
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + E * threadIdx.x;
#pragma unroll
    for (int i = 0; i < R; ++i)
      w[i] = n > E * kWidth * i ? p[E * kWidth * i] | static_cast<uint32_t>(p[E * kWidth * i + 1]) << 16 : 0u;
  }
}
template <typename T, int kWidth, int R>
__device__ __forceinline__ void write_words(const uint32_t (&w)[R], uint8_t* row, int n) {
  constexpr int E = Word<T>::kElems;
  if (E == 1 || !(reinterpret_cast<uintptr_t>(row) & 2)) {
    uint32_t* p = reinterpret_cast<uint32_t*>(row) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (n > E * kWidth * i) p[kWidth * i] = w[i];
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(row) + E * threadIdx.x;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (n > E * kWidth * i) {
        p[E * kWidth * i] = static_cast<uint16_t>(w[i]);
        p[E * kWidth * i + 1] = static_cast<uint16_t>(w[i] >> 16);
      }
  }
}

// Every buffer has a spare element behind the row's place, zero in the input
// buffers, so that the last word of a row of 16-bit elements may be half.
template <typename T, int kOut, int kWidth, int R>
__global__ void __launch_bounds__(kWidth, staged_resident(kWidth, R)) mla_norm_staged_kernel(const NormParams p) {
  extern __shared__ __align__(16) uint8_t buffers[];
  __shared__ float slots[2][32];
  constexpr int E = Word<T>::kElems, kSize = sizeof(T), kOutSize = kOut == MLA_NORM_OUT_SAME ? kSize : 1;
  using Bits = typename std::conditional<kSize == 2, uint16_t, uint32_t>::type;
  const int t = threadIdx.x, bytes = p.cols * kSize, buffer = staged_buffer(p.cols, kSize);
  const int n = p.cols - E * t;   // elements from the thread's first word to the row's end
  uint8_t* const sum_s = buffers + (p.residual ? 4 : 2) * buffer;   // residual_out's lines, then out's
  uint8_t* const out_s = sum_s + (p.residual_out ? buffer : 0);
  auto stage = [&](int s, int which) { return buffers + (p.residual ? 2 * s + which : s) * buffer; };
  // The lines of a row into a buffer; its ends' elements into a register.
  auto fetch = [&](const Lines& l, uint8_t* to) {
    const uint8_t* from = l.line + 16 * t;
    to += 16 * t;
#pragma unroll
    for (int i = 0; i <= R / 4; ++i)   // 4 R kWidth bytes at most
      if (t + kWidth * i >= l.first && t + kWidth * i < l.end) cp_async_16(to + 16 * kWidth * i, from + 16 * kWidth * i, 16);
    Bits v = 0;
    if (t < 32) {
      const int at = l.edge(t, kSize, bytes);
      if (at >= 0) v = *reinterpret_cast<const Bits*>(l.line + at);
    }
    return v;
  };
  auto put_edge = [&](const Lines& l, uint8_t* to, Bits v) {
    if (t >= 32) return;
    const int at = l.edge(t, kSize, bytes);
    if (at >= 0) *reinterpret_cast<Bits*>(to + at) = v;
    if (t == 0) *reinterpret_cast<Bits*>(to + l.shift + bytes) = 0;
  };
  auto flush = [&](const Lines& l, const uint8_t* from, auto size) {
    constexpr int z = decltype(size)::value;
    using B = typename std::conditional<z == 1, uint8_t, typename std::conditional<z == 2, uint16_t, uint32_t>::type>::type;
    uint8_t* to = l.line + 16 * t;
#pragma unroll
    for (int i = 0; i <= R * z / (4 * kSize); ++i)
      if (t + kWidth * i >= l.first && t + kWidth * i < l.end)
        *reinterpret_cast<uint4*>(to + 16 * kWidth * i) = *reinterpret_cast<const uint4*>(from + 16 * (t + kWidth * i));
    if (t < 32) {
      const int at = l.edge(t, z, p.cols * z);
      if (at >= 0) *reinterpret_cast<B*>(l.line + at) = *reinterpret_cast<const B*>(from + at);
    }
  };
  after_predecessor();
  float w[R * E];
#pragma unroll
  for (int i = 0; i < R * E; ++i) {
    const int c = (t + i / E * kWidth) * E + i % E;
    w[i] = p.weight && c < p.cols ? to_f32(static_cast<const T*>(p.weight)[c]) : 1.f;
  }
  // the rows' addresses, a step of gridDim rows from one to the next
  const int64_t row0 = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row0 * p.x_stride;
  const T* r = static_cast<const T*>(p.residual) + row0 * p.residual_stride;
  T* ro = static_cast<T*>(p.residual_out) + row0 * p.residual_out_stride;
  uint8_t* y = static_cast<uint8_t*>(p.out) + row0 * p.out_stride * kOutSize;
  const int64_t x_step = gridDim.x * p.x_stride, r_step = gridDim.x * p.residual_stride;
  const int64_t ro_step = gridDim.x * p.residual_out_stride, y_step = gridDim.x * p.out_stride * kOutSize;
  Lines xl(x, bytes), rl(r, bytes);
  Bits x_edge = fetch(xl, stage(0, 0)), r_edge = p.residual ? fetch(rl, stage(0, 1)) : static_cast<Bits>(0);
  cp_async_commit();
  int s = 0;
  for (int64_t row = row0; row < p.rows; row += gridDim.x, s ^= 1, ro += ro_step, y += y_step) {
    const int x_shift = xl.shift, r_shift = rl.shift;
    put_edge(xl, stage(s, 0), x_edge);
    if (p.residual) put_edge(rl, stage(s, 1), r_edge);
    // the next row, into buffers that were read before the last row's sums met
    if (row + gridDim.x < p.rows) {
      x += x_step;
      xl = Lines(x, bytes);
      x_edge = fetch(xl, stage(s ^ 1, 0));
      if (p.residual) {
        r += r_step;
        rl = Lines(r, bytes);
        r_edge = fetch(rl, stage(s ^ 1, 1));
      }
    }
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    uint32_t words[R];
    float h[R * E];
    read_words<T, kWidth>(words, stage(s, 0) + x_shift, n);
#pragma unroll
    for (int i = 0; i < R; ++i) Word<T>::get(words[i], h + i * E);
    if (p.residual) {
      read_words<T, kWidth>(words, stage(s, 1) + r_shift, n);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float b[E];
        Word<T>::get(words[i], b);
#pragma unroll
        for (int j = 0; j < E; ++j) h[i * E + j] += b[j];
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < R * E; ++i) sum = fmaf(h[i], h[i], sum);
    const Lines ol(ro, bytes);
    if (p.residual_out) {
#pragma unroll
      for (int i = 0; i < R; ++i) words[i] = Word<T>::put(h + i * E);
      write_words<T, kWidth>(words, sum_s + ol.shift, n);
    }
    const float rstd = rsqrt_exact(row_reduce<0, false>(sum, slots[0]) * p.inv_cols + p.eps);
    if (p.residual_out) flush(ol, sum_s, std::integral_constant<int, kSize>());
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < R * E; ++i) {
      h[i] = norm_product<kOut>(h[i], rstd, w[i]);   // elements that are not there: 0, or like all others where rstd is not finite
      if (kOut == MLA_NORM_OUT_E4M3_ROW) amax = max_nan(amax, fabsf(h[i]));
    }
    const Lines yl(y, p.cols * kOutSize);
    uint8_t* ys = out_s + yl.shift;
    if (kOut == MLA_NORM_OUT_SAME) {
#pragma unroll
      for (int i = 0; i < R; ++i) words[i] = Word<T>::put(h + i * E);
      write_words<T, kWidth>(words, ys, n);
    } else {
      float inv = 1.f;
      if (kOut == MLA_NORM_OUT_E4M3_ROW) {
        const float scale = max_nan(row_reduce<0, true>(amax, slots[1]) * (1.f / 448.f), kMinRowScale);
        inv = 1.f / scale;
        if (t == 0) static_cast<float*>(p.scales)[row] = scale;
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float* v = h + i * E;
        bool some = true;
        if (kOut == MLA_NORM_OUT_E4M3_E8M0) {   // a group is 32 / E neighbouring lanes' words
          float a = 0.f;
#pragma unroll
          for (int j = 0; j < E; ++j) a = fmaxf(a, fabsf(v[j]));
#pragma unroll
          for (int o = 16 / E; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
          some = a > 0.f;
          const uint32_t byte = e4m3_scale_byte(a);
          inv = scale_byte_reciprocal(byte);
          if (n > E * kWidth * i && t % (32 / E) == 0)
            static_cast<uint8_t*>(p.scales)[row * p.scale_stride + (t + kWidth * i) * E / 32] = static_cast<uint8_t>(byte);
        }
        words[i] = e4m3x2(v[0] * inv, v[E - 1] * inv);
        if (!some) words[i] &= 0x7F7Fu;   // zeros without their signs (or NaN)
      }
      if (E == 2 && !(reinterpret_cast<uintptr_t>(ys) & 1)) {
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (n > E * kWidth * i) reinterpret_cast<uint16_t*>(ys)[t + kWidth * i] = static_cast<uint16_t>(words[i]);
      } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (n > E * kWidth * i) {
            ys[E * (t + kWidth * i)] = static_cast<uint8_t>(words[i]);
            if (E == 2) ys[E * (t + kWidth * i) + 1] = static_cast<uint8_t>(words[i] >> 8);
          }
      }
    }
    __syncthreads();
    flush(yl, out_s, std::integral_constant<int, kOutSize>());
  }
}

template <typename T, int kOut, bool kWords, int R, int G>
cudaError_t launch_one(const NormParams& p, int threads, cudaStream_t stream) {
  constexpr int kRows = G == 0 ? 1 : kRowThreads / (G == 0 ? 1 : G);
  const int blocks = p.rows / kRows + (p.rows % kRows != 0);
  auto launch = [&](auto kernel, int t) { return launch_dependent(kernel, blocks, t, 0, stream, p); };
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

template <typename T, int kOut, int kWidth, int R>
cudaError_t launch_staged(const NormParams& p, cudaStream_t stream) {
  const int buffer = staged_buffer(p.cols, sizeof(T));
  const int smem = buffer * ((p.residual ? 4 : 2) + (p.residual_out ? 1 : 0)) +
                   staged_buffer(p.cols, kOut == MLA_NORM_OUT_SAME ? sizeof(T) : 1);
  auto kernel = mla_norm_staged_kernel<T, kOut, kWidth, R>;
  if (smem > 48 * 1024) {
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
  }
  const int fit = 232448 / (smem + 2048);   // and as far as shared memory goes
  const int blocks = 152 * (fit < staged_resident(kWidth, R) ? fit : staged_resident(kWidth, R));
  return launch_dependent(kernel, p.rows < blocks ? p.rows : blocks, kWidth, smem, stream, p);
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
  const int words = (p.cols + Word<T>::kElems - 1) / Word<T>::kElems;
  if (many && words > 128 && words <= 4096) {
    if (words <= 512) return launch_staged<T, kOut, 128, 4>(p, stream);
    if (words <= 1024) return launch_staged<T, kOut, 128, 8>(p, stream);
    if (words <= 1536) return launch_staged<T, kOut, 128, 12>(p, stream);
    if (words <= 2048) return launch_staged<T, kOut, 128, 16>(p, stream);
    return launch_staged<T, kOut, 256, 16>(p, stream);
  }
  constexpr int kMost = sizeof(T) == 4 ? 32 : 16;   // words of a thread
  if (words <= 128) return launch_one<T, kOut, true, 4, 32>(p, 0, stream);
  if (words <= 4096) return launch_one<T, kOut, true, 4, 0>(p, threads(words, 4), stream);
  return launch_one<T, kOut, true, kMost, 0>(p, threads(words, kMost), stream);
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
