// The paged latent cache, many tokens at a time: the append (latent norm, key
// rotation, quantisation on the way) and the gather back to dense bf16 rows.
// One warp per token in both.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "mla_layer_internal.h"
#include "mla_quant.cuh"
#include "mla_rows.cuh"
#include "mla_turn.cuh"
#include "sm103_ptx.cuh"

namespace mla {

namespace {

constexpr int kTokenWarps = 4;
// Tokens a warp takes one after another, at most: the append's warps keep the
// norm's weights and the rotation's table, the gather's only their slots (100,011
// rows normed and rotated into FP8: 4 37.9, 8 36.0, 16 37.4 us, into bf16 37.9, 37.2,
// 39.3; 204,800 rows out of FP8: 2 66.9, 4 61.4, 8 62.8, 16 66.3 us).
constexpr int kAppendChunk = 8, kGatherChunk = 4;

// The slot of token t in the pool: -1 where the token is to be left alone
// (negative position), -2 where it has none (which is reported).
__device__ __forceinline__ int32_t token_slot(const TokenParams& p, int32_t t, int32_t pos) {
  if (pos < 0) return -1;
  const int32_t r = p.requests ? p.requests[t] : t / p.per_request;
  uint32_t bad = 0;
  int32_t page = 0;
  const int32_t index = pos >> p.page_shift;
  if (r < 0 || r >= p.batch || index >= p.max_pages) {
    bad = MLA_STATUS_BAD_INDEX;
  } else {
    page = p.block_table[static_cast<int64_t>(r) * p.max_pages + index];
    if (page < 0 || page >= p.num_pages) bad = MLA_STATUS_BAD_PAGE;
  }
  if (bad) {
    if (p.status) atomicOr(p.status, bad);
    return -2;
  }
  return (page << p.page_shift) + (pos & ((1 << p.page_shift) - 1));   // below 2^31: checked by the host
}

// A warp's tokens: `chunk` consecutive ones, their slots found side by side,
// lane l holding token first + l's.
struct WarpTokens {
  int32_t first, count, pos, slot;
  __device__ __forceinline__ WarpTokens(const TokenParams& p, int32_t chunk) {
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * kTokenWarps + (threadIdx.x >> 5)) * chunk;
    first = static_cast<int32_t>(min(at, static_cast<int64_t>(p.tokens)));
    count = min(chunk, p.tokens - first);
  }
  __device__ __forceinline__ void find(const TokenParams& p, int lane) {
    pos = lane < count ? p.positions[first + lane] : -1;
    slot = token_slot(p, first + lane, pos);
  }
};

// Maximum over aligned sets of kLanes lanes.
template <int kLanes>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float abs_max(const float2 (&v)[4]) {
  float m = max3(fabsf(v[0].x), fabsf(v[0].y), fabsf(v[1].x));
  m = max3(m, fabsf(v[1].y), fabsf(v[2].x));
  m = max3(m, fabsf(v[2].y), fabsf(v[3].x));
  return max3(m, fabsf(v[3].y), 0.f);   // 0 where all are NaN
}

constexpr int kStageBytes = 640;   // a 594-byte row behind a shift of at most 14

// kBytes of a row, laid out in shared memory as they lie around the row's
// 16-byte boundaries (`shift` bytes into the first line), to global memory:
// whole 16-byte lines, and the row's ends in units of kUnit bytes, which
// divides its address.  A warp writes a row.
template <int kBytes, int kUnit>
__device__ __forceinline__ void write_row(uint8_t* dst, const uint8_t* stage, int shift, int lane) {
  using Unit = typename std::conditional<kUnit == 2, uint16_t, uint32_t>::type;
  constexpr int kSide = 16 / kUnit;                       // lanes for each end
  const int first = (shift + 15) >> 4, end = (shift + kBytes) >> 4;   // whole lines: kBytes / 16 or one less
  uint4* lines = reinterpret_cast<uint4*>(dst - shift);
  const uint4* from = reinterpret_cast<const uint4*>(stage);
  if (lane >= first && lane < end) lines[lane] = from[lane];
  if (kBytes > 32 * 16 && 32 + lane < end) lines[32 + lane] = from[32 + lane];
  const int at = lane < kSide ? shift + kUnit * lane : 16 * end + kUnit * (lane - kSide);
  if (lane < 2 * kSide && at < (lane < kSide ? 16 * first : shift + kBytes))
    *reinterpret_cast<Unit*>(dst - shift + at) = *reinterpret_cast<const Unit*>(stage + at);
}

// One warp per token at a time.  A row costs 1,152 bytes read and 1,152, 594
// or 324 written; 100,011 rows of 2,688 bytes' stride with norm and rotation take
// 36.0 us into FP8 (4.9 TB/s), 35.9 into FP4, 37.2 into bf16 (6.2 TB/s), and without
// 29.2, 25.8 and 36.2.  Into bf16 memory bounds the kernel; into the quantised
// caches it is the warp's own chain of shuffles, stage and write-out: 295 (FP8)
// and 300 (FP4) instructions a row issue in 70 % of the cycles, with at most 28
// warps on a multiprocessor, 203 and 211 without norm and rotation.  So every
// value stays in its lane, one shuffle reduction gives the norm, the cosine and
// sine are one pair per lane, arithmetic goes in pairs, slots are found one token
// per lane, the next rows are on their way while one is computed (copied
// asynchronously into the lane's own places in a ring in shared memory: loads into
// registers were moved behind the arithmetic by the compiler, 37 -> 60 us when it
// was tried), and norm and rotation are compiled in or out.
constexpr int kRing = 3;   // rows of a warp on their way or in use

template <int kKv, bool kNorm, bool kRotate>
__global__ void __launch_bounds__(32 * kTokenWarps, 7)
    mla_append_tokens_kernel(const __grid_constant__ AppendTokensParams p, const int32_t chunk) {
  __shared__ __align__(16) uint8_t ring_s[kTokenWarps][kRing][kDqk * 2];
  __shared__ __align__(16) uint8_t stage_s[kKv == MLA_KV_BF16 ? 1 : kTokenWarps][kStageBytes];
  const int lane = threadIdx.x & 31;
  after_predecessor();
  WarpTokens tok(p.t, chunk);
  if (tok.count <= 0) return;
  const uint8_t* src = reinterpret_cast<const uint8_t*>(p.rows + tok.first * p.row_stride) + 16 * lane;
  uint8_t* const ring = ring_s[threadIdx.x >> 5][0] + 16 * lane;
  auto fetch = [&](int j) {   // each lane the pieces that it will read
    if (j < tok.count) {
      uint8_t* to = ring + (j % kRing) * (kDqk * 2);
      cp_async_16(to, src, 16);
      cp_async_16(to + 512, src + 512, 16);
      cp_async_4(to + 2 * kDc - 12 * lane, src + 2 * kDc - 12 * lane);
      src += 2 * p.row_stride;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int j = 0; j < kRing - 1; ++j) fetch(j);
  tok.find(p.t, lane);   // a chain of three loads, beside the rows
  const uint64_t turns = kRotate ? p.table.turns[lane] : 0;
  const float amplitude = p.table.amplitude;
  const bool halves = p.table.halves != 0;
  float2 w[8];
  if (kNorm) {
    const uint4 a = reinterpret_cast<const uint4*>(p.weight)[lane], b = reinterpret_cast<const uint4*>(p.weight)[32 + lane];
    const uint32_t words[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = make_float2(bf16_lo(words[i]), bf16_hi(words[i]));
  }
  uint8_t* const stage = stage_s[kKv == MLA_KV_BF16 ? 0 : threadIdx.x >> 5];
  for (int j = 0; j < tok.count; ++j) {
    fetch(j + kRing - 1);
    const int32_t pos = __shfl_sync(0xffffffffu, tok.pos, j), at = __shfl_sync(0xffffffffu, tok.slot, j);
    cp_async_wait<kRing - 1>();
    if (at < 0) continue;
    const int64_t slot = at;
    const uint8_t* in = ring + (j % kRing) * (kDqk * 2);
    RowWords row;
    row.a = *reinterpret_cast<const uint4*>(in);
    row.b = *reinterpret_cast<const uint4*>(in + 512);
    row.key = *reinterpret_cast<const uint32_t*>(in + 2 * kDc - 12 * lane);
    const uint32_t words[8] = {row.a.x, row.a.y, row.a.z, row.a.w, row.b.x, row.b.y, row.b.z, row.b.w};
    float2 y[2][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i >> 2][i & 3] = make_float2(bf16_lo(words[i]), bf16_hi(words[i]));
    auto norm = [&] {
      float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum2 = __ffma2_rn(y[i >> 2][i & 3], y[i >> 2][i & 3], sum2);
      float sum = sum2.x + sum2.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float mean = sum * (1.f / kDc) + p.eps;
      float rstd = rsqrtf(mean);
      // Below 2^-100 (0x0D800000), infinite or NaN: squares out of the range of 32
      // bits are summed again, the row scaled by a power of two (rare; see row_rstd
      // of the norm).
      if (__float_as_uint(mean) - 0x0D800000u >= 0x7F800000u - 0x0D800000u) {
        const bool small = mean < 0x1p-100f;
        const float f = small ? 0x1p100f : 0x1p-34f, g = small ? 1.f : 0x1p-38f;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float2& v = y[i >> 2][i & 3];
          asm volatile("{\n .reg .f32 v;\n mul.f32 %0, %0, %3;\n mul.f32 v, %0, %4;\n fma.rn.f32 %2, v, v, %2;\n"
                       " mul.f32 %1, %1, %3;\n mul.f32 v, %1, %4;\n fma.rn.f32 %2, v, v, %2;\n}"
                       : "+f"(v.x), "+f"(v.y), "+f"(sum)
                       : "f"(f), "f"(g));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        rstd = rsqrtf(sum * (1.f / kDc) + p.eps * f * g * f * g) * g;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        y[i >> 2][i & 3] = __fmul2_rn(__fmul2_rn(y[i >> 2][i & 3], make_float2(rstd, rstd)), w[i]);
    };
    float2 k = make_float2(bf16_lo(row.key), bf16_hi(row.key));
    auto turn = [&] {
      float c, s;
      turn_cos_sin(turns, pos, &c, &s);
      c *= amplitude;
      s *= amplitude;
      if (halves) {   // value l of both halves to lane l, and back
        const float a0 = __shfl_sync(0xffffffffu, k.x, lane >> 1), a1 = __shfl_sync(0xffffffffu, k.y, lane >> 1);
        const float b0 = __shfl_sync(0xffffffffu, k.x, 16 + (lane >> 1)), b1 = __shfl_sync(0xffffffffu, k.y, 16 + (lane >> 1));
        const float a = lane & 1 ? a1 : a0, b = lane & 1 ? b1 : b0;
        const float ya = a * c - b * s, yb = a * s + b * c;
        const int from = (2 * lane) & 31;
        const float ra0 = __shfl_sync(0xffffffffu, ya, from), ra1 = __shfl_sync(0xffffffffu, ya, from + 1);
        const float rb0 = __shfl_sync(0xffffffffu, yb, from), rb1 = __shfl_sync(0xffffffffu, yb, from + 1);
        k = lane < 16 ? make_float2(ra0, ra1) : make_float2(rb0, rb1);
      } else {
        k = make_float2(k.x * c - k.y * s, k.x * s + k.y * c);
      }
    };
    // The norm's branch is a border for the compiler: the rotation before it hides
    // the row's loads and sum (100,011 rows into FP8 36.0 us, behind it 36.9), but
    // in FP4 keeps more alive (with the gather 66.6, behind it 61.5).
    constexpr bool kTurnFirst = kKv != MLA_KV_FP4_E2M1_E8M0;
    if (kRotate && kTurnFirst) turn();
    if (kNorm) norm();
    if (kRotate && !kTurnFirst) turn();
    if (kKv == MLA_KV_BF16) {
      uint8_t* dst = p.kv + slot * (kDqk * 2);
      uint4 oa = row.a, ob = row.b;   // as they came without a norm
      if (kNorm) {
        oa = make_uint4(pack_bf16(y[0][0]), pack_bf16(y[0][1]), pack_bf16(y[0][2]), pack_bf16(y[0][3]));
        ob = make_uint4(pack_bf16(y[1][0]), pack_bf16(y[1][1]), pack_bf16(y[1][2]), pack_bf16(y[1][3]));
      }
      reinterpret_cast<uint4*>(dst)[lane] = oa;
      reinterpret_cast<uint4*>(dst)[32 + lane] = ob;
      reinterpret_cast<uint32_t*>(dst + kDc * 2)[lane] = kRotate ? pack_bf16(k) : row.key;
      continue;
    }
    constexpr bool kFp8 = kKv == MLA_KV_FP8_E4M3_E8M0;
    constexpr int kGroup = kFp8 ? 4 : 2;   // lanes of a group of the latent; of the key four times as many
    const float m[2] = {lanes_max<kGroup>(abs_max(y[0])), lanes_max<kGroup>(abs_max(y[1]))};
    const float mk = lanes_max<4 * kGroup>(max3(fabsf(k.x), fabsf(k.y), 0.f));
    uint32_t e[2] = {kFp8 ? e4m3_scale_byte(m[0]) : e2m1_scale_byte(m[0]),
                     kFp8 ? e4m3_scale_byte(m[1]) : e2m1_scale_byte(m[1])};
    uint32_t ek = kFp8 ? e4m3_scale_byte(mk) : e2m1_scale_byte(mk);
    // y / 2^e; a group of zeros gets codes 0 whatever their signs, which adding
    // +0 does there, and adding -0 changes nothing elsewhere.  A NaN stays one.
    auto scaled = [](float2 v, uint32_t byte, float amax) {
      const float inv = scale_byte_reciprocal(byte), sign = amax == 0.f ? 0.f : -0.f;
      return __ffma2_rn(v, make_float2(inv, inv), make_float2(sign, sign));
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i >> 2][i & 3] = scaled(y[i >> 2][i & 3], e[i >> 2], m[i >> 2]);
    const float2 yk = scaled(k, ek, mk);
    constexpr int kRow = kFp8 ? kFp8RowBytes : kFp4RowBytes, kCodes = kFp8 ? kDqk : kFp4CodeBytes;
    uint8_t* dst = p.kv + slot * kRow;
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(dst) & 15);   // even; a multiple of 4 in FP4
    uint8_t* st = stage + shift;
    if (kFp8) {
      __syncwarp();
      uint16_t* st2 = reinterpret_cast<uint16_t*>(st);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        st2[(i >> 2) * 128 + 4 * lane + (i & 3)] = static_cast<uint16_t>(e4m3x2(y[i >> 2][i & 3].x, y[i >> 2][i & 3].y));
      st2[256 + lane] = static_cast<uint16_t>(e4m3x2(yk.x, yk.y));
    } else {
      const uint32_t c[2] = {pack_e2m1(y[0]), pack_e2m1(y[1])}, ck = pack_e2m1(yk);
      // a sum of magnitudes is NaN where a value is (they are at most 6, or infinite)
      float nan = fabsf(k.x) + fabsf(k.y);
#pragma unroll
      for (int i = 0; i < 8; ++i) nan += fabsf(y[i >> 2][i & 3].x) + fabsf(y[i >> 2][i & 3].y);
      if (__any_sync(0xffffffffu, nan != nan)) {   // rare: NaN groups get the NaN scale
        bool n[2] = {false, false};
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i >> 2] |= y[i >> 2][i & 3].x != y[i >> 2][i & 3].x || y[i >> 2][i & 3].y != y[i >> 2][i & 3].y;
        const uint32_t nan0 = __ballot_sync(0xffffffffu, n[0]) >> (lane & ~1) & 3u;
        const uint32_t nan1 = __ballot_sync(0xffffffffu, n[1]) >> (lane & ~1) & 3u;
        const uint32_t nank = __ballot_sync(0xffffffffu, k.x != k.x || k.y != k.y) >> (lane & ~7) & 0xFFu;
        if (nan0) e[0] = 255;
        if (nan1) e[1] = 255;
        if (nank) ek = 255;
      }
      __syncwarp();
      reinterpret_cast<uint32_t*>(st)[lane] = c[0];
      reinterpret_cast<uint32_t*>(st)[32 + lane] = c[1];
      st[256 + lane] = static_cast<uint8_t>(ck);
    }
    if (lane % kGroup == 0) {
      st[kCodes + lane / kGroup] = static_cast<uint8_t>(e[0]);
      st[kCodes + 32 / kGroup + lane / kGroup] = static_cast<uint8_t>(e[1]);
    }
    if (lane % (4 * kGroup) == 0) st[kCodes + 64 / kGroup + lane / (4 * kGroup)] = static_cast<uint8_t>(ek);
    __syncwarp();
    write_row<kRow, kFp8 ? 2 : 4>(dst, stage, shift, lane);
  }
}

// One warp per token at a time.  Bound by memory: a cached row read, 1,152
// bytes written.  Slots are found one token per lane, so that the chain
// position -> page -> row is walked once for a warp's tokens, and two rows are
// on their way at a time.  204,800 rows out of FP8 61.4 us: the 236 MB written
// alone take 61.3 us at the 3.85 TB/s of a plain fill; out of FP4 52.2, out of
// bf16 71.4 us (6.64 TB/s, 0.98 of the copy rate).
template <int kKv>
__global__ void __launch_bounds__(32 * kTokenWarps)
    mla_gather_kernel(const __grid_constant__ GatherParams p, const int32_t chunk) {
  const int lane = threadIdx.x & 31;
  after_predecessor();
  WarpTokens tok(p.t, chunk);
  tok.find(p.t, lane);
  for (int j = 0; j < tok.count; j += 2) {
    CachedRow<kKv> c[2];
    int32_t slot[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      slot[i] = j + i < tok.count ? __shfl_sync(0xffffffffu, tok.slot, j + i) : -1;
      if (slot[i] >= 0) load_cached(&c[i], p.kv, slot[i], lane);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (slot[i] == -1) continue;
      RowWords r = {};
      if (slot[i] >= 0) r = cached_to_bf16(c[i], slot[i]);
      uint16_t* out = p.out + (tok.first + j + i) * p.out_stride;
      reinterpret_cast<uint4*>(out)[lane] = r.a;
      reinterpret_cast<uint4*>(out)[32 + lane] = r.b;
      reinterpret_cast<uint32_t*>(out + kDc)[lane] = r.key;
    }
  }
}

// Tokens of a warp: one while there are multiprocessors to fill (latency),
// then up to `most` as the warps get to more than fit at once.
int chunk_of(int32_t tokens, int most) {
  const int c = tokens / (kSms * 32);
  return c < 1 ? 1 : c > most ? most : c;
}
int blocks_of(int32_t tokens, int chunk) {
  return static_cast<int>((static_cast<int64_t>(tokens) + kTokenWarps * chunk - 1) / (kTokenWarps * chunk));
}

}  // namespace

namespace {

template <int kKv>
cudaError_t launch_append_into(const AppendTokensParams& p, cudaStream_t stream) {
  const int chunk = chunk_of(p.t.tokens, kAppendChunk), blocks = blocks_of(p.t.tokens, chunk);
  auto launch = [&](auto kernel) { return launch_dependent(kernel, blocks, 32 * kTokenWarps, 0, stream, p, chunk); };
  if (p.weight)
    return p.rotate ? launch(mla_append_tokens_kernel<kKv, true, true>) : launch(mla_append_tokens_kernel<kKv, true, false>);
  return p.rotate ? launch(mla_append_tokens_kernel<kKv, false, true>) : launch(mla_append_tokens_kernel<kKv, false, false>);
}

}  // namespace

cudaError_t launch_append_tokens(const AppendTokensParams& p, cudaStream_t stream) {
  if (p.t.tokens == 0) return cudaSuccess;
  if (p.t.kv_dtype == MLA_KV_BF16) return launch_append_into<MLA_KV_BF16>(p, stream);
  if (p.t.kv_dtype == MLA_KV_FP8_E4M3_E8M0) return launch_append_into<MLA_KV_FP8_E4M3_E8M0>(p, stream);
  return launch_append_into<MLA_KV_FP4_E2M1_E8M0>(p, stream);
}

cudaError_t launch_gather(const GatherParams& p, cudaStream_t stream) {
  if (p.t.tokens == 0) return cudaSuccess;
  const int chunk = chunk_of(p.t.tokens, kGatherChunk), blocks = blocks_of(p.t.tokens, chunk);
  const int threads = 32 * kTokenWarps;
  if (p.t.kv_dtype == MLA_KV_BF16)
    return launch_dependent(mla_gather_kernel<MLA_KV_BF16>, blocks, threads, 0, stream, p, chunk);
  if (p.t.kv_dtype == MLA_KV_FP8_E4M3_E8M0)
    return launch_dependent(mla_gather_kernel<MLA_KV_FP8_E4M3_E8M0>, blocks, threads, 0, stream, p, chunk);
  return launch_dependent(mla_gather_kernel<MLA_KV_FP4_E2M1_E8M0>, blocks, threads, 0, stream, p, chunk);
}

}  // namespace mla
