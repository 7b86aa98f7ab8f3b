// The paged latent cache, many tokens at a time: the append (latent norm, key
// rotation, quantisation on the way) and the gather back to dense bf16 rows.
// One warp per token in both.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mla_layer_internal.h"
#include "mla_quant.cuh"
#include "mla_turn.cuh"

namespace mla {

namespace {

constexpr int kTokenWarps = 4;

// The slot of token t in the pool, -1 where the token is to be left alone
// (negative position) and -2 where it has none (reported by lane 0).
__device__ __forceinline__ int64_t token_slot(const TokenParams& p, int64_t t, int32_t pos, bool report) {
  if (pos < 0) return -1;
  const int32_t r = p.requests ? p.requests[t] : static_cast<int32_t>(t / p.per_request);
  uint32_t bad = 0;
  int32_t page = 0;
  if (r < 0 || r >= p.batch || pos >= static_cast<int64_t>(p.max_pages) * p.page_size) {
    bad = MLA_STATUS_BAD_INDEX;
  } else {
    page = p.block_table[static_cast<int64_t>(r) * p.max_pages + pos / p.page_size];
    if (page < 0 || page >= p.num_pages) bad = MLA_STATUS_BAD_PAGE;
  }
  if (bad) {
    if (report && p.status) atomicOr(p.status, bad);
    return -2;
  }
  return static_cast<int64_t>(page) * p.page_size + pos % p.page_size;
}

__device__ __forceinline__ uint16_t f32_to_bf16_bits(float v) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&h);
}

__global__ void __launch_bounds__(32 * kTokenWarps) mla_append_tokens_kernel(const __grid_constant__ AppendTokensParams p) {
  __shared__ float row_s[kTokenWarps][kDqk];
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokenWarps + (threadIdx.x >> 5);
  if (t >= p.t.tokens) return;
  const int32_t pos = p.t.positions[t];
  const int64_t slot = token_slot(p.t, t, pos, lane == 0);
  if (slot < 0) return;
  float* row = row_s[threadIdx.x >> 5];
  const uint16_t* src = p.rows + t * p.row_stride;
  float sum = 0.f;
  for (int c = lane; c < kDqk; c += 32) {
    const float v = bf16_bits_to_f32(src[c]);
    row[c] = v;
    if (c < kDc) sum = fmaf(v, v, sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncwarp();
  if (p.weight) {
    const float rstd = rsqrtf(sum * (1.f / kDc) + p.eps);
    for (int c = lane; c < kDc; c += 32) row[c] = row[c] * rstd * bf16_bits_to_f32(p.weight[c]);
  }
  if (p.rotate) {
    const int a = kDc + (p.table.halves ? lane : 2 * lane), b = a + (p.table.halves ? 32 : 1);
    float cs, sn;
    turn_cos_sin(p.table.turns[lane], pos, &cs, &sn);
    cs *= p.table.amplitude;
    sn *= p.table.amplitude;
    const float va = row[a], vb = row[b];
    row[a] = va * cs - vb * sn;
    row[b] = va * sn + vb * cs;
  }
  __syncwarp();
  if (p.t.kv_dtype == MLA_KV_BF16) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(p.kv) + slot * kDqk;
    for (int c = lane; c < kDqk; c += 32) dst[c] = f32_to_bf16_bits(row[c]);
    return;
  }
  const bool fp8 = p.t.kv_dtype == MLA_KV_FP8_E4M3_E8M0;
  uint8_t* dst = p.kv + slot * (fp8 ? kFp8RowBytes : kFp4RowBytes);
  for (int c = lane; c < kDqk; c += 32) {
    const float v = row[c];
    float amax = fabsf(v);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (fp8) {
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
      const int e = amax > 0.f ? max(-127, min(127, ceil_log2_over_448(amax))) : -127;
      dst[c] = static_cast<uint8_t>(amax > 0.f || v != v ? f32_to_e4m3(v * pow2_neg(e)) : 0u);
      if (lane == 0) dst[kDqk + (c >> 5)] = static_cast<uint8_t>(e + 127);
    } else {
      const uint32_t nans = __ballot_sync(0xffffffffu, v != v) & (lane < 16 ? 0xFFFFu : 0xFFFF0000u);
      const int e = amax > 0.f ? max(-127, min(127, ceil_log2_over_6(amax))) : -127;
      const uint32_t code = amax > 0.f ? f32_to_e2m1(v * pow2_neg(e)) : 0u;
      const uint32_t hi = __shfl_down_sync(0xffffffffu, code, 1);
      if ((lane & 1) == 0) dst[c >> 1] = static_cast<uint8_t>(code | (hi << 4));
      if ((lane & 15) == 0) dst[kFp4CodeBytes + (c >> 4)] = static_cast<uint8_t>(nans ? 255 : e + 127);
    }
  }
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t code) {
  uint32_t two;
  const uint16_t in = static_cast<uint16_t>(code);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(in));
  return __half2float(__ushort_as_half(static_cast<uint16_t>(two & 0xFFFFu)));
}

// 2^(s - 127) of a scale byte, NaN for 255.
__device__ __forceinline__ float e8m0_to_f32(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FFFFFFFu : s << 23);
}

__device__ __forceinline__ float e2m1_to_f32(uint32_t code) {
  const uint32_t m = code & 7u;
  const float a = m < 2 ? 0.5f * m : static_cast<float>(2 + (m & 1u)) * static_cast<float>(1u << ((m >> 1) - 1)) * 0.5f;
  return code & 8u ? -a : a;
}

__global__ void __launch_bounds__(32 * kTokenWarps) mla_gather_kernel(const GatherParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokenWarps + (threadIdx.x >> 5);
  if (t >= p.t.tokens) return;
  const int64_t slot = token_slot(p.t, t, p.t.positions[t], lane == 0);
  if (slot == -1) return;
  uint16_t* out = p.out + t * p.out_stride;
  if (slot < 0) {
    for (int c = lane; c < kDqk; c += 32) out[c] = 0;
  } else if (p.t.kv_dtype == MLA_KV_BF16) {
    const uint16_t* src = reinterpret_cast<const uint16_t*>(p.kv) + slot * kDqk;
    for (int c = lane; c < kDqk; c += 32) out[c] = src[c];
  } else if (p.t.kv_dtype == MLA_KV_FP8_E4M3_E8M0) {
    const uint8_t* src = p.kv + slot * kFp8RowBytes;
    for (int c = lane; c < kDqk; c += 32)
      out[c] = f32_to_bf16_bits(e4m3_to_f32(src[c]) * e8m0_to_f32(src[kDqk + (c >> 5)]));
  } else {
    const uint8_t* src = p.kv + slot * kFp4RowBytes;
    for (int c = lane; c < kDqk; c += 32)
      out[c] = f32_to_bf16_bits(e2m1_to_f32((src[c >> 1] >> (4 * (c & 1))) & 15u) *
                                e8m0_to_f32(src[kFp4CodeBytes + (c >> 4)]));
  }
}

int blocks_of(int32_t tokens) { return tokens / kTokenWarps + (tokens % kTokenWarps != 0); }

}  // namespace

cudaError_t launch_append_tokens(const AppendTokensParams& p, cudaStream_t stream) {
  if (p.t.tokens == 0) return cudaSuccess;
  mla_append_tokens_kernel<<<blocks_of(p.t.tokens), 32 * kTokenWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_gather(const GatherParams& p, cudaStream_t stream) {
  if (p.t.tokens == 0) return cudaSuccess;
  mla_gather_kernel<<<blocks_of(p.t.tokens), 32 * kTokenWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
