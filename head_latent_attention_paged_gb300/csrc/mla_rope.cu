// Rotary positions on part of each head.
//
// Bound by memory: the rotated part of every head is read and written once.
// A block takes a few tokens; one thread per (token, pair) computes the cosine
// and sine into shared memory, from where all heads of the token use them, so
// the functions cost one evaluation per token and pair.  The heads are then
// units of 16 bytes (one piece, or in the half layout a piece of each half;
// single pairs where the addresses do not allow that), a thread's first units
// being loaded before the cosines are computed.
#include <cuda_runtime.h>

#include "mla_layer_internal.h"
#include "mla_turn.cuh"
#include "mla_types.cuh"

namespace mla {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnits = 4;       // units a thread has in flight
constexpr int kRopeMaxTokens = 16;  // tokens of a block

// n / d for n < 2^31, as a multiplication (round-up method).
struct Divider {
  uint32_t d, mul, shift;
  explicit Divider(uint32_t div) : d(div) {
    uint32_t l = 0;
    while (l < 32 && (1ull << l) < div) ++l;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - div)) / div + 1);
    shift = l;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return (__umulhi(n, mul) + n) >> shift;   // no carry: n < 2^31
  }
};

struct RopeLaunch {
  RopeParams p;
  int32_t block_tokens;             // tokens of a block
  int32_t turn_units;               // of a head: rotated units, then copied ones
  Divider units, heads;             // units of a head, heads
};

template <int kBytes>
struct Piece;
template <>
struct Piece<16> { using type = uint4; };
template <>
struct Piece<4> { using type = uint32_t; };
template <>
struct Piece<2> { using type = uint16_t; };

template <typename T, int kVec>
union Elems {
  typename Piece<sizeof(T) * kVec>::type raw;
  T v[kVec];
  __device__ Elems() {}
};

template <typename T, int kVec, bool kHalves>
__global__ void __launch_bounds__(kRopeThreads) mla_rope_kernel(const __grid_constant__ RopeLaunch a) {
  extern __shared__ float2 cs[];    // [block_tokens][pairs], then the tokens' positions
  const RopeParams& p = a.p;
  using E = Elems<T, kVec>;
  using Raw = decltype(E::raw);
  // a rotated unit: kPieces pieces, kPairs pairs
  constexpr bool kTwo = kVec == 1 || kHalves;
  constexpr int kPieces = kTwo ? 2 : 1, kPairs = kTwo ? kVec : kVec / 2;
  const int pairs = p.dim >> 1;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.block_tokens;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(a.block_tokens), p.tokens - t0));
  int32_t* pos_s = reinterpret_cast<int32_t*>(cs + a.block_tokens * pairs);
  const uint32_t items = static_cast<uint32_t>(tokens) * a.units.d * a.heads.d;
  const T* x = static_cast<const T*>(p.x);
  T* out = static_cast<T*>(p.out);
  E e[kRopeUnits][kPieces];
  // where unit k lies: token of the block, head, first element (-1: none) and
  // for a rotated unit its first pair
  struct Place {
    int32_t token, element, pair;
    int64_t head;
  };
  auto place = [&](uint32_t k) {
    Place q;
    const uint32_t th = a.units.div(k), u = k - th * a.units.d, tok = a.heads.div(th);
    q.token = static_cast<int32_t>(tok);
    q.head = th - tok * a.heads.d;
    q.pair = -1;
    if (static_cast<int32_t>(u) < a.turn_units) {
      q.pair = u * kPairs;
      q.element = p.offset + (kVec == 1 && !kHalves ? 2 * u : u * kVec);
    } else {
      const int32_t c = (u - a.turn_units) * kVec;
      q.element = c < p.offset ? c : c + p.dim;
    }
    return q;
  };
  const int second = kHalves ? pairs : 1;   // elements to a unit's second piece
  auto load = [&](uint32_t k0) {
#pragma unroll
    for (int i = 0; i < kRopeUnits; ++i) {
      const uint32_t k = k0 + i * kRopeThreads;
      if (k >= items) continue;
      const Place q = place(k);
      const T* src = x + (t0 + q.token) * p.x_token_stride + q.head * p.x_head_stride + q.element;
      e[i][0].raw = *reinterpret_cast<const Raw*>(src);
      if (kTwo && q.pair >= 0) e[i][kPieces - 1].raw = *reinterpret_cast<const Raw*>(src + second);
    }
  };
  load(threadIdx.x);
  for (int i = threadIdx.x; i < tokens * pairs; i += kRopeThreads) {
    const int tok = i / pairs;
    const int32_t pos = p.positions[t0 + tok];
    float c, s;
    turn_cos_sin(p.table.turns[i - tok * pairs], pos, &c, &s);
    cs[i] = make_float2(c * p.table.amplitude, (p.transposed ? -s : s) * p.table.amplitude);
    if (i == tok * pairs) pos_s[tok] = pos;
  }
  __syncthreads();
  for (uint32_t k0 = threadIdx.x; k0 < items; k0 += kRopeUnits * kRopeThreads) {
#pragma unroll
    for (int i = 0; i < kRopeUnits; ++i) {
      const uint32_t k = k0 + i * kRopeThreads;
      if (k >= items) continue;
      const Place q = place(k);
      if (pos_s[q.token] < 0) continue;
      T* dst = out + (t0 + q.token) * p.out_token_stride + q.head * p.out_head_stride + q.element;
      if (q.pair >= 0) {
        const float2* f = cs + q.token * pairs + q.pair;
        E y[kPieces];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const float2 g = f[j];
          const float va = to_f32(kTwo ? e[i][0].v[j % kVec] : e[i][0].v[2 * j % kVec]);
          const float vb = to_f32(kTwo ? e[i][kPieces - 1].v[j % kVec] : e[i][0].v[(2 * j + 1) % kVec]);
          const T ya = from_f32<T>(va * g.x - vb * g.y), yb = from_f32<T>(va * g.y + vb * g.x);
          if (kTwo) {
            y[0].v[j % kVec] = ya;
            y[kPieces - 1].v[j % kVec] = yb;
          } else {
            y[0].v[2 * j % kVec] = ya;
            y[0].v[(2 * j + 1) % kVec] = yb;
          }
        }
        *reinterpret_cast<Raw*>(dst) = y[0].raw;
        if (kTwo) *reinterpret_cast<Raw*>(dst + second) = y[kPieces - 1].raw;
      } else {
        *reinterpret_cast<Raw*>(dst) = e[i][0].raw;
      }
    }
    if (k0 + kRopeUnits * kRopeThreads < items) load(k0 + kRopeUnits * kRopeThreads);
  }
}

template <typename T, int kVec>
cudaError_t launch_vec(const RopeParams& p, cudaStream_t stream) {
  const bool halves = p.table.halves != 0;
  const int per_turn = kVec == 1 ? 2 : halves ? 2 * kVec : kVec;   // elements of a rotated unit
  const int turn_units = p.dim / per_turn;
  const int copied = p.x == p.out ? 0 : (p.head_dim - p.dim) / kVec;
  const int64_t per_token = static_cast<int64_t>(p.heads) * (turn_units + copied);
  // tokens of a block: enough units to keep its threads busy, as long as
  // that leaves two blocks for each multiprocessor
  int64_t tokens = (2 * kRopeUnits * kRopeThreads + per_token - 1) / per_token;
  if (tokens > p.tokens / (2 * 152)) tokens = p.tokens / (2 * 152);
  if (tokens > kRopeMaxTokens) tokens = kRopeMaxTokens;
  if (tokens < 1) tokens = 1;
  RopeLaunch a{p, static_cast<int32_t>(tokens), turn_units, Divider(turn_units + copied), Divider(p.heads)};
  const int blocks = static_cast<int>((p.tokens + tokens - 1) / tokens);
  const int smem = static_cast<int>(tokens) * (p.dim / 2 * 8 + 4);
  if (halves)
    mla_rope_kernel<T, kVec, true><<<blocks, kRopeThreads, smem, stream>>>(a);
  else
    mla_rope_kernel<T, kVec, false><<<blocks, kRopeThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const RopeParams& p, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  auto fits = [&](const void* base, int64_t token_stride, int64_t head_stride) {
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && token_stride % V == 0 && head_stride % V == 0;
  };
  const bool vec = p.offset % V == 0 && p.dim % (p.table.halves ? 2 * V : V) == 0 &&
                   (p.x == p.out || p.head_dim % V == 0) && fits(p.x, p.x_token_stride, p.x_head_stride) &&
                   fits(p.out, p.out_token_stride, p.out_head_stride);
  return vec ? launch_vec<T, V>(p, stream) : launch_vec<T, 1>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  if (p.tokens == 0) return cudaSuccess;
  if (p.dtype == MLA_DTYPE_BF16) return launch_typed<__nv_bfloat16>(p, stream);
  if (p.dtype == MLA_DTYPE_F16) return launch_typed<__half>(p, stream);
  return launch_typed<float>(p, stream);
}

}  // namespace mla
