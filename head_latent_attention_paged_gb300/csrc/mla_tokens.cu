// The paged latent cache, many tokens at a time: the append (latent norm, key
// rotation, quantisation on the way) and the gather back to dense bf16 rows.
// One warp per token in both.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "mla_layer_internal.h"
#include "mla_quant.cuh"
#include "mla_turn.cuh"

namespace mla {

namespace {

constexpr int kTokenWarps = 4;
constexpr int kAppendBlocks = 152 * 8;   // resident blocks: each warp then takes further tokens

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

// Two bf16 of a word, as f32.
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// e4m3 codes of two values, the first in the low byte; e2m1 codes of two, the
// first in the low nibble.  Nearest even, saturating, as f32_to_e4m3 and
// f32_to_e2m1.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(hi), "f"(lo));
  return two;
}
__device__ __forceinline__ uint32_t pack_e2m1(float lo, float hi) {
  uint32_t two;
  asm("{\n .reg .b8 c;\n cvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n cvt.u32.u8 %0, c;\n}"
      : "=r"(two)
      : "f"(hi), "f"(lo));
  return two;
}

// The warp's row: lane l holds latent values 8 l .. 8 l + 7 and 256 + 8 l ..,
// and key values 2 l and 2 l + 1.
struct RowWords {
  uint4 a, b;
  uint32_t key;
};

__device__ __forceinline__ void load_row(RowWords* r, const uint16_t* src, int lane) {
  const uint4* s4 = reinterpret_cast<const uint4*>(src);
  r->a = s4[lane];
  r->b = s4[32 + lane];
  r->key = reinterpret_cast<const uint32_t*>(src + kDc)[lane];
}

// Maximum over aligned sets of `lanes` lanes.
__device__ __forceinline__ float lanes_max(float v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <bool kFp8>
__device__ __forceinline__ int group_exponent(float amax) {
  if (!(amax > 0.f)) return -127;
  return max(-127, min(127, kFp8 ? ceil_log2_over_448(amax) : ceil_log2_over_6(amax)));
}

constexpr int kStageBytes = 640;   // a 594-byte row behind a shift of at most 14

// One warp per token at a time.  Bound by memory (a 1,152-byte row read, a
// 1,152-, 594- or 324-byte row written) where the instructions for a row's
// norm, rotation and codes can be kept near 250: every value stays in its
// lane, one shuffle reduction gives the norm, the cosine and sine are one pair
// per lane, and the next row is on its way while one is computed.
template <int kKv>
__global__ void __launch_bounds__(32 * kTokenWarps) mla_append_tokens_kernel(const __grid_constant__ AppendTokensParams p) {
  __shared__ __align__(16) uint8_t stage_s[kKv == MLA_KV_FP8_E4M3_E8M0 ? kTokenWarps : 1][kStageBytes];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTokenWarps;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kTokenWarps + warp;
  if (t >= p.t.tokens) return;
  RowWords next;
  int32_t next_pos = p.t.positions[t];
  load_row(&next, p.rows + t * p.row_stride, lane);
  const uint64_t turns = p.rotate ? p.table.turns[lane] : 0;
  uint4 wa = {}, wb = {};
  if (p.weight) {
    wa = reinterpret_cast<const uint4*>(p.weight)[lane];
    wb = reinterpret_cast<const uint4*>(p.weight)[32 + lane];
  }
  for (; t < p.t.tokens; t += stride) {
    const RowWords row = next;
    const int32_t pos = next_pos;
    if (t + stride < p.t.tokens) {
      next_pos = p.t.positions[t + stride];
      load_row(&next, p.rows + (t + stride) * p.row_stride, lane);
    }
    const int64_t slot = token_slot(p.t, t, pos, lane == 0);
    if (slot < 0) continue;
    const uint32_t words[8] = {row.a.x, row.a.y, row.a.z, row.a.w, row.b.x, row.b.y, row.b.z, row.b.w};
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[2 * i] = bf16_lo(words[i]);
      y[2 * i + 1] = bf16_hi(words[i]);
    }
    if (p.weight) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) sum = fmaf(y[i], y[i], sum);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float rstd = rsqrtf(sum * (1.f / kDc) + p.eps);
      const uint32_t w[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[2 * i] = y[2 * i] * rstd * bf16_lo(w[i]);
        y[2 * i + 1] = y[2 * i + 1] * rstd * bf16_hi(w[i]);
      }
    }
    float k0 = bf16_lo(row.key), k1 = bf16_hi(row.key);
    if (p.rotate) {
      float c, s;
      turn_cos_sin(turns, pos, &c, &s);
      c *= p.table.amplitude;
      s *= p.table.amplitude;
      if (p.table.halves) {   // value l of both halves to lane l, and back
        const float a0 = __shfl_sync(0xffffffffu, k0, lane >> 1), a1 = __shfl_sync(0xffffffffu, k1, lane >> 1);
        const float b0 = __shfl_sync(0xffffffffu, k0, 16 + (lane >> 1)), b1 = __shfl_sync(0xffffffffu, k1, 16 + (lane >> 1));
        const float a = lane & 1 ? a1 : a0, b = lane & 1 ? b1 : b0;
        const float ya = a * c - b * s, yb = a * s + b * c;
        const int from = (2 * lane) & 31;
        const float ra0 = __shfl_sync(0xffffffffu, ya, from), ra1 = __shfl_sync(0xffffffffu, ya, from + 1);
        const float rb0 = __shfl_sync(0xffffffffu, yb, from), rb1 = __shfl_sync(0xffffffffu, yb, from + 1);
        k0 = lane < 16 ? ra0 : rb0;
        k1 = lane < 16 ? ra1 : rb1;
      } else {
        const float a = k0, b = k1;
        k0 = a * c - b * s;
        k1 = a * s + b * c;
      }
    }
    if (kKv == MLA_KV_BF16) {
      uint8_t* dst = p.kv + slot * (kDqk * 2);
      uint4 oa = row.a, ob = row.b;   // as they came without a norm
      if (p.weight) {
        oa = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        ob = make_uint4(pack_bf16(y[8], y[9]), pack_bf16(y[10], y[11]), pack_bf16(y[12], y[13]), pack_bf16(y[14], y[15]));
      }
      reinterpret_cast<uint4*>(dst)[lane] = oa;
      reinterpret_cast<uint4*>(dst)[32 + lane] = ob;
      reinterpret_cast<uint32_t*>(dst + kDc * 2)[lane] = p.rotate ? pack_bf16(k0, k1) : row.key;
      continue;
    }
    constexpr bool kFp8 = kKv == MLA_KV_FP8_E4M3_E8M0;
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m0 = fmaxf(m0, fabsf(y[i]));
      m1 = fmaxf(m1, fabsf(y[8 + i]));
    }
    // a group is 4 lanes of 8 values and 16 lanes of 2 (FP8), 2 and 8 (FP4)
    m0 = lanes_max(m0, kFp8 ? 4 : 2);
    m1 = lanes_max(m1, kFp8 ? 4 : 2);
    const float mk = lanes_max(fmaxf(fabsf(k0), fabsf(k1)), kFp8 ? 16 : 8);
    const int e0 = group_exponent<kFp8>(m0), e1 = group_exponent<kFp8>(m1), ek = group_exponent<kFp8>(mk);
    const float s0 = pow2_neg(e0), s1 = pow2_neg(e1), sk = pow2_neg(ek);
    // A group of zeros has codes 0 whatever their signs; a NaN stays one.
    if (kFp8) {
      uint32_t code[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        code[i] = pack_e4m3(y[2 * i] * s0, y[2 * i + 1] * s0);
        code[4 + i] = pack_e4m3(y[8 + 2 * i] * s1, y[9 + 2 * i] * s1);
      }
      uint32_t kcode = pack_e4m3(k0 * sk, k1 * sk);
      // with amax 0 every code is a signed zero (0x00, 0x80) or NaN (0x7F, 0xFF)
      auto unsign = [](uint32_t c) { return (c & 0x7F7Fu); };
      if (m0 == 0.f)
        for (int i = 0; i < 4; ++i) code[i] = unsign(code[i]);
      if (m1 == 0.f)
        for (int i = 4; i < 8; ++i) code[i] = unsign(code[i]);
      if (mk == 0.f) kcode = unsign(kcode);
      // The row starts on any even address: it is laid out in shared memory at
      // the same place within 16 bytes and leaves in 16-byte stores, its ends
      // in pairs of bytes.
      uint8_t* dst = p.kv + slot * kFp8RowBytes;
      const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(dst) & 15);
      uint8_t* st = stage_s[warp];
      uint16_t* st2 = reinterpret_cast<uint16_t*>(st + shift);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        st2[4 * lane + i] = static_cast<uint16_t>(code[i]);
        st2[128 + 4 * lane + i] = static_cast<uint16_t>(code[4 + i]);
      }
      st2[256 + lane] = static_cast<uint16_t>(kcode);
      if ((lane & 3) == 0) {
        st[shift + kDqk + (lane >> 2)] = static_cast<uint8_t>(e0 + 127);
        st[shift + kDqk + 8 + (lane >> 2)] = static_cast<uint8_t>(e1 + 127);
      }
      if ((lane & 15) == 0) st[shift + kDqk + 16 + (lane >> 4)] = static_cast<uint8_t>(ek + 127);
      __syncwarp();
      const int first = shift ? 1 : 0, end = (shift + kFp8RowBytes) >> 4;   // whole pieces
      uint8_t* base = dst - shift;
      for (int j = first + lane; j < end; j += 32)
        reinterpret_cast<uint4*>(base)[j] = reinterpret_cast<const uint4*>(st)[j];
      const int head = (16 * first - shift) >> 1;                            // pairs before them
      const int tail = (shift + kFp8RowBytes - 16 * end) >> 1;               // and behind
      const int at = lane < 8 ? (lane < head ? lane : -1)
                              : (lane - 8 < tail ? 8 * end - (shift >> 1) + lane - 8 : -1);
      if (lane < 16 && at >= 0) reinterpret_cast<uint16_t*>(dst)[at] = st2[at];
    } else {
      uint32_t c0 = 0, c1 = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c0 |= pack_e2m1(y[2 * i] * s0, y[2 * i + 1] * s0) << (8 * i);
        c1 |= pack_e2m1(y[8 + 2 * i] * s1, y[9 + 2 * i] * s1) << (8 * i);
      }
      uint32_t ck = pack_e2m1(k0 * sk, k1 * sk);
      bool n0 = false, n1 = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n0 |= y[i] != y[i];
        n1 |= y[8 + i] != y[8 + i];
      }
      // groups with a NaN get the NaN scale
      const uint32_t nan0 = __ballot_sync(0xffffffffu, n0) >> (lane & ~1) & 3u;
      const uint32_t nan1 = __ballot_sync(0xffffffffu, n1) >> (lane & ~1) & 3u;
      const uint32_t nank = __ballot_sync(0xffffffffu, k0 != k0 || k1 != k1) >> (lane & ~7) & 0xFFu;
      if (m0 == 0.f) c0 = 0;
      if (m1 == 0.f) c1 = 0;
      if (mk == 0.f) ck = 0;
      uint8_t* dst = p.kv + slot * kFp4RowBytes;   // rows start on 4 bytes
      reinterpret_cast<uint32_t*>(dst)[lane] = c0;
      reinterpret_cast<uint32_t*>(dst)[32 + lane] = c1;
      dst[256 + lane] = static_cast<uint8_t>(ck);
      if ((lane & 1) == 0) {
        dst[kFp4CodeBytes + (lane >> 1)] = static_cast<uint8_t>(nan0 ? 255 : e0 + 127);
        dst[kFp4CodeBytes + 16 + (lane >> 1)] = static_cast<uint8_t>(nan1 ? 255 : e1 + 127);
      }
      if ((lane & 7) == 0) dst[kFp4CodeBytes + 32 + (lane >> 3)] = static_cast<uint8_t>(nank ? 255 : ek + 127);
    }
  }
}

// 2^(s - 127) of a scale byte, NaN for 255.
__device__ __forceinline__ float e8m0_to_f32(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FFFFFFFu : s << 23);
}

// Two e4m3 codes (two e2m1 codes in a byte), the first in the low bits, times
// a scale, as two bf16.  Both convert to f16 exactly and the product is
// rounded once.
__device__ __forceinline__ uint32_t scaled_bf16(uint32_t f16x2, float scale) {
  const __half2 h = *reinterpret_cast<const __half2*>(&f16x2);
  return pack_bf16(__low2float(h) * scale, __high2float(h) * scale);
}
__device__ __forceinline__ uint32_t e4m3x2_to_bf16(uint32_t codes, float scale) {
  uint32_t two;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(static_cast<uint16_t>(codes)));
  return scaled_bf16(two, scale);
}
__device__ __forceinline__ uint32_t e2m1x2_to_bf16(uint32_t codes, float scale) {
  uint32_t two;
  asm("{\n .reg .b8 c;\n cvt.u8.u32 c, %1;\n cvt.rn.f16x2.e2m1x2 %0, c;\n}" : "=r"(two) : "r"(codes));
  return scaled_bf16(two, scale);
}

// One warp per token.  Bound by memory: a cached row read, 1,152 bytes
// written.  Lanes hold the row as in the append (RowWords).
template <int kKv>
__global__ void __launch_bounds__(32 * kTokenWarps) mla_gather_kernel(const GatherParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokenWarps + (threadIdx.x >> 5);
  if (t >= p.t.tokens) return;
  const int64_t slot = token_slot(p.t, t, p.t.positions[t], lane == 0);
  if (slot == -1) return;
  RowWords r = {};
  if (slot >= 0) {
    if (kKv == MLA_KV_BF16) {
      load_row(&r, reinterpret_cast<const uint16_t*>(p.kv) + slot * kDqk, lane);
    } else if (kKv == MLA_KV_FP8_E4M3_E8M0) {
      // rows start on even addresses: aligned words, shifted by two bytes
      // where the row starts between them
      const uint8_t* src = p.kv + slot * kFp8RowBytes;
      const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 2);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(src - odd) + 2 * lane;
      uint32_t a0 = w[0], a1 = w[1], b0 = w[64], b1 = w[65];
      if (odd) {
        const uint32_t a2 = w[2], b2 = w[66];
        a0 = __funnelshift_r(a0, a1, 16);
        a1 = __funnelshift_r(a1, a2, 16);
        b0 = __funnelshift_r(b0, b1, 16);
        b1 = __funnelshift_r(b1, b2, 16);
      }
      const uint32_t k = reinterpret_cast<const uint16_t*>(src + kDc)[lane];
      const float s0 = e8m0_to_f32(src[kDqk + (lane >> 2)]), s1 = e8m0_to_f32(src[kDqk + 8 + (lane >> 2)]);
      const float sk = e8m0_to_f32(src[kDqk + 16 + (lane >> 4)]);
      r.a = make_uint4(e4m3x2_to_bf16(a0, s0), e4m3x2_to_bf16(a0 >> 16, s0), e4m3x2_to_bf16(a1, s0),
                       e4m3x2_to_bf16(a1 >> 16, s0));
      r.b = make_uint4(e4m3x2_to_bf16(b0, s1), e4m3x2_to_bf16(b0 >> 16, s1), e4m3x2_to_bf16(b1, s1),
                       e4m3x2_to_bf16(b1 >> 16, s1));
      r.key = e4m3x2_to_bf16(k, sk);
    } else {
      const uint8_t* src = p.kv + slot * kFp4RowBytes;   // rows start on 4 bytes
      const uint32_t a = reinterpret_cast<const uint32_t*>(src)[lane], b = reinterpret_cast<const uint32_t*>(src)[32 + lane];
      const uint32_t k = src[256 + lane];
      const float s0 = e8m0_to_f32(src[kFp4CodeBytes + (lane >> 1)]), s1 = e8m0_to_f32(src[kFp4CodeBytes + 16 + (lane >> 1)]);
      const float sk = e8m0_to_f32(src[kFp4CodeBytes + 32 + (lane >> 3)]);
      r.a = make_uint4(e2m1x2_to_bf16(a & 255u, s0), e2m1x2_to_bf16(a >> 8 & 255u, s0),
                       e2m1x2_to_bf16(a >> 16 & 255u, s0), e2m1x2_to_bf16(a >> 24, s0));
      r.b = make_uint4(e2m1x2_to_bf16(b & 255u, s1), e2m1x2_to_bf16(b >> 8 & 255u, s1),
                       e2m1x2_to_bf16(b >> 16 & 255u, s1), e2m1x2_to_bf16(b >> 24, s1));
      r.key = e2m1x2_to_bf16(k, sk);
    }
  }
  uint16_t* out = p.out + t * p.out_stride;
  reinterpret_cast<uint4*>(out)[lane] = r.a;
  reinterpret_cast<uint4*>(out)[32 + lane] = r.b;
  reinterpret_cast<uint32_t*>(out + kDc)[lane] = r.key;
}

int blocks_of(int32_t tokens) { return tokens / kTokenWarps + (tokens % kTokenWarps != 0); }

}  // namespace

cudaError_t launch_append_tokens(const AppendTokensParams& p, cudaStream_t stream) {
  if (p.t.tokens == 0) return cudaSuccess;
  const int blocks = min(blocks_of(p.t.tokens), kAppendBlocks);
  if (p.t.kv_dtype == MLA_KV_BF16)
    mla_append_tokens_kernel<MLA_KV_BF16><<<blocks, 32 * kTokenWarps, 0, stream>>>(p);
  else if (p.t.kv_dtype == MLA_KV_FP8_E4M3_E8M0)
    mla_append_tokens_kernel<MLA_KV_FP8_E4M3_E8M0><<<blocks, 32 * kTokenWarps, 0, stream>>>(p);
  else
    mla_append_tokens_kernel<MLA_KV_FP4_E2M1_E8M0><<<blocks, 32 * kTokenWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_gather(const GatherParams& p, cudaStream_t stream) {
  if (p.t.tokens == 0) return cudaSuccess;
  const int blocks = blocks_of(p.t.tokens);
  if (p.t.kv_dtype == MLA_KV_BF16)
    mla_gather_kernel<MLA_KV_BF16><<<blocks, 32 * kTokenWarps, 0, stream>>>(p);
  else if (p.t.kv_dtype == MLA_KV_FP8_E4M3_E8M0)
    mla_gather_kernel<MLA_KV_FP8_E4M3_E8M0><<<blocks, 32 * kTokenWarps, 0, stream>>>(p);
  else
    mla_gather_kernel<MLA_KV_FP4_E2M1_E8M0><<<blocks, 32 * kTokenWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
