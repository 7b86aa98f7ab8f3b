// Cached rows of every format as a warp holds them: loads of a row's bytes and
// their values as bf16, exact but for bf16's own range.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "mla_internal.h"

namespace mla {

// Two bf16 of a word, as f32.
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
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

// 2^(s - 127) of a scale byte, NaN for 255.
__device__ __forceinline__ float e8m0_to_f32(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FFFFFFFu : s << 23);
}

// Two e4m3 codes (two e2m1 codes in a byte), the first in the low bits, times
// a scale, as two bf16.  Both convert to f16 exactly and the product is
// rounded once.
__device__ __forceinline__ uint32_t scaled_bf16(uint32_t f16x2, float scale) {
  const __half2 h = *reinterpret_cast<const __half2*>(&f16x2);
  return pack_bf16(__fmul2_rn(__half22float2(h), make_float2(scale, scale)));
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

// A cached row's bytes as its warp loads them: lanes as in RowWords.
template <int kKv>
struct CachedRow {
  RowWords bf16;                // MLA_KV_BF16
  uint32_t a[3], b[3], key;     // codes: FP8 in words from the aligned one at
  uint32_t sa, sb, sk;          // or before the lane's first; scale bytes
};

template <int kKv>
__device__ __forceinline__ void load_cached(CachedRow<kKv>* r, const uint8_t* kv, int64_t slot, int lane) {
  if (kKv == MLA_KV_BF16) {
    load_row(&r->bf16, reinterpret_cast<const uint16_t*>(kv) + slot * kDqk, lane);
  } else if (kKv == MLA_KV_FP8_E4M3_E8M0) {
    const uint8_t* src = kv + slot * kFp8RowBytes;
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 2);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(src - odd) + 2 * lane;
    r->a[0] = w[0];
    r->a[1] = w[1];
    r->b[0] = w[64];
    r->b[1] = w[65];
    if (odd) {
      r->a[2] = w[2];
      r->b[2] = w[66];
    }
    r->key = reinterpret_cast<const uint16_t*>(src + kDc)[lane];
    r->sa = src[kDqk + (lane >> 2)];
    r->sb = src[kDqk + 8 + (lane >> 2)];
    r->sk = src[kDqk + 16 + (lane >> 4)];
  } else {
    const uint8_t* src = kv + slot * kFp4RowBytes;   // rows start on 4 bytes
    r->a[0] = reinterpret_cast<const uint32_t*>(src)[lane];
    r->b[0] = reinterpret_cast<const uint32_t*>(src)[32 + lane];
    r->key = src[256 + lane];
    r->sa = src[kFp4CodeBytes + (lane >> 1)];
    r->sb = src[kFp4CodeBytes + 16 + (lane >> 1)];
    r->sk = src[kFp4CodeBytes + 32 + (lane >> 3)];
  }
}

template <int kKv>
__device__ __forceinline__ RowWords cached_to_bf16(const CachedRow<kKv>& c, int64_t slot) {
  if (kKv == MLA_KV_BF16) return c.bf16;
  RowWords r;
  const float sa = e8m0_to_f32(c.sa), sb = e8m0_to_f32(c.sb), sk = e8m0_to_f32(c.sk);
  if (kKv == MLA_KV_FP8_E4M3_E8M0) {
    // a row of an odd slot starts two bytes into its first word (the pool
    // starts on 16 bytes, a row has 594)
    uint32_t a0 = c.a[0], a1 = c.a[1], b0 = c.b[0], b1 = c.b[1];
    if (slot & 1) {
      a0 = __funnelshift_r(a0, a1, 16);
      a1 = __funnelshift_r(a1, c.a[2], 16);
      b0 = __funnelshift_r(b0, b1, 16);
      b1 = __funnelshift_r(b1, c.b[2], 16);
    }
    r.a = make_uint4(e4m3x2_to_bf16(a0, sa), e4m3x2_to_bf16(a0 >> 16, sa), e4m3x2_to_bf16(a1, sa),
                     e4m3x2_to_bf16(a1 >> 16, sa));
    r.b = make_uint4(e4m3x2_to_bf16(b0, sb), e4m3x2_to_bf16(b0 >> 16, sb), e4m3x2_to_bf16(b1, sb),
                     e4m3x2_to_bf16(b1 >> 16, sb));
    r.key = e4m3x2_to_bf16(c.key, sk);
  } else {
    const uint32_t a = c.a[0], b = c.b[0];
    r.a = make_uint4(e2m1x2_to_bf16(a & 255u, sa), e2m1x2_to_bf16(a >> 8 & 255u, sa),
                     e2m1x2_to_bf16(a >> 16 & 255u, sa), e2m1x2_to_bf16(a >> 24, sa));
    r.b = make_uint4(e2m1x2_to_bf16(b & 255u, sb), e2m1x2_to_bf16(b >> 8 & 255u, sb),
                     e2m1x2_to_bf16(b >> 16 & 255u, sb), e2m1x2_to_bf16(b >> 24, sb));
    r.key = e2m1x2_to_bf16(c.key, sk);
  }
  return r;
}

}  // namespace mla
