// Rotary positions on part of each head.
//
// Bound by memory: the rotated part of every head is read and written once.
// A head's rotated part is cut into units of 16 bytes (in the half layout 16
// bytes of each half; single pairs where the addresses do not allow that).  A
// thread owns one unit's place within the head for some heads of one token: it
// sets their loads going, computes the unit's few cosines and sines meanwhile
// and uses them for all its heads, so only the table goes through shared memory
// and no thread waits for another's values.  32,768 tokens of 20 heads, 64 of
// 256 turned in place, 27.6 us: 6.1 TB/s in pieces of 128 bytes every 512 (27.1
// us where the turned parts lie side by side).
#include <cuda_runtime.h>

#include "mla_layer_internal.h"
#include "mla_turn.cuh"
#include "mla_types.cuh"

namespace mla {

namespace {

// 32,768 tokens of 20 heads (64 of 256, bf16) and 4,099 of 8 (96 of 128, f32,
// halves, out of place): 4 heads in flight and up to 12 28.0 and 6.1 us, up to 8
// 28.3 and 6.1, up to 20 29.0 and 6.1; 2 and 12 29.5 and 6.7; blocks of 256 28.3
// and 6.3; cosines shared through shared memory 35 and 10.4.
constexpr int kRopeThreads = 128;
constexpr int kRopeHeads = 4;       // heads a thread has in flight
constexpr int kRopeMostHeads = 12;  // and takes altogether
// Threads to have before they take more heads each: 639 tokens of 45 heads (128
// of 256) with 512, 768 and 1,024 for each multiprocessor 3.1, 3.6 and 4.1 us, 333
// of 29 (192, f32, halves) 3.5, 3.1 and 4.6.  A thread with eight cosines (bf16
// halves) counts as four: 2,688 of 11 (64 of 256) 2.6 us, as one 4.0.
constexpr int64_t kRopeFill = 152 * 768;

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
  uint32_t turn_all, all;           // its threads' places: rotated units of all its tokens' heads, then
                                    // copied ones, so that few warps have both (out of place 42,129 tokens of
                                    // one head, 96 of 192: head by head 13.5 us, so 12.7; 352 of 51 heads,
                                    // 128 of 256: 4.6 and 4.2)
  Divider turns, copies, groups;    // of a head: rotated and copied units; threads sharing a token's heads
};

// One access of kVec elements: 16 bytes, or a single element.
template <typename T, int kVec>
struct Access {
  uint4 raw;
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = raw; }
  __device__ __forceinline__ void get(float* v) const { unpack16<T>(raw, v); }
  __device__ __forceinline__ void put(const float* v) { raw = pack16<T>(v); }
};
template <typename T>
struct Access<T, 1> {
  T raw;
  __device__ __forceinline__ void load(const T* p) { raw = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = raw; }
  __device__ __forceinline__ void get(float* v) const { v[0] = to_f32(raw); }
  __device__ __forceinline__ void put(const float* v) { raw = from_f32<T>(v[0]); }
};

template <typename T, int kVec, bool kHalves, int kHeads>
__global__ void __launch_bounds__(kRopeThreads) mla_rope_kernel(const __grid_constant__ RopeLaunch a) {
  const RopeParams& p = a.p;
  using E = Access<T, kVec>;
  // a rotated unit: kPieces pieces, kPairs pairs
  constexpr bool kTwo = kVec == 1 || kHalves;
  constexpr int kPieces = kTwo ? 2 : 1, kPairs = kTwo ? kVec : kVec / 2;
  // The table to shared memory: a warp's lanes read many of its entries, one
  // after another where they are parameters (45 heads of 128 turned, 639 tokens:
  // 6.0 -> 4.1 us).  It is there before the predecessor's end.
  __shared__ uint64_t turns[MLA_ROPE_MAX_DIM / 2];
  for (int i = threadIdx.x; i < p.dim >> 1; i += kRopeThreads) turns[i] = p.table.turns[i];
  __syncthreads();
  after_predecessor();
  for (uint32_t k = blockIdx.y * kRopeThreads + threadIdx.x; k < a.all; k += gridDim.y * kRopeThreads) {
    const bool turn = k < a.turn_all;
    const Divider& units = turn ? a.turns : a.copies;
    const uint32_t at = turn ? k : k - a.turn_all, row = units.div(at), u = at - row * units.d;
    const uint32_t tok = a.groups.div(row), group = row - tok * a.groups.d;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * a.block_tokens + tok;
    if (t >= p.tokens) continue;
    // on its way beside the first heads where registers allow: units of one
    // piece (a decode step 1.85 -> 1.67 us; units of two 22.5 -> 23.8 for 8192 x 32
    // heads of 128)
    const int32_t pos = p.positions[t];
    if (kTwo && pos < 0) continue;
    int32_t element;
    if (turn) {
      element = p.offset + (kVec == 1 && !kHalves ? 2 * u : u * kVec);
    } else {
      const int32_t c = u * kVec;
      element = c < p.offset ? c : c + p.dim;
    }
    const int second = kHalves ? p.dim >> 1 : 1;   // elements to a unit's second piece
    const int64_t x_step = static_cast<int64_t>(a.groups.d) * p.x_head_stride;
    const int64_t out_step = static_cast<int64_t>(a.groups.d) * p.out_head_stride;
    const T* src = static_cast<const T*>(p.x) + t * p.x_token_stride +
                   static_cast<int64_t>(group) * p.x_head_stride + element;
    T* dst = static_cast<T*>(p.out) + t * p.out_token_stride +
             static_cast<int64_t>(group) * p.out_head_stride + element;
    float c[kPairs], s[kPairs];
    bool ready = false;
    for (int32_t h = group; h < p.heads; h += kHeads * a.groups.d) {
      E e[kHeads][kPieces];
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        if (h + i * static_cast<int32_t>(a.groups.d) >= p.heads) continue;
        e[i][0].load(src + i * x_step);
        if (kTwo && turn) e[i][kPieces - 1].load(src + i * x_step + second);
      }
      if (pos < 0) break;
      if (turn && !ready) {
        ready = true;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          turn_cos_sin(turns[u * kPairs + j], pos, &c[j], &s[j]);
          c[j] *= p.table.amplitude;
          s[j] *= p.transposed ? -p.table.amplitude : p.table.amplitude;
        }
      }
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        if (h + i * static_cast<int32_t>(a.groups.d) >= p.heads) continue;
        if (turn) {
          float v[kPieces * kVec];
#pragma unroll
          for (int j = 0; j < kPieces; ++j) e[i][j].get(v + j * kVec);
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            float& va = v[kTwo ? j : 2 * j];
            float& vb = v[kTwo ? kVec + j : 2 * j + 1];
            const float ya = va * c[j] - vb * s[j], yb = va * s[j] + vb * c[j];
            va = ya;
            vb = yb;
          }
          e[i][0].put(v);
          if (kTwo) {
            e[i][kPieces - 1].put(v + (kPieces - 1) * kVec);
            e[i][kPieces - 1].store(dst + i * out_step + second);
          }
        }
        e[i][0].store(dst + i * out_step);
      }
      src += kHeads * x_step;
      dst += kHeads * out_step;
    }
  }
}

template <typename T, int kVec>
cudaError_t launch_vec(const RopeParams& p, cudaStream_t stream) {
  const bool halves = p.table.halves != 0;
  const int per_turn = kVec == 1 ? 2 : halves ? 2 * kVec : kVec;   // elements of a rotated unit
  const int turn_units = p.dim / per_turn;
  const int copies = p.x == p.out ? 0 : (p.head_dim - p.dim) / kVec, units = turn_units + copies;
  // threads that share a token's heads: the fewer, the more heads use a
  // thread's cosines, as long as there are threads to fill the
  // multiprocessors
  const int64_t one = static_cast<int64_t>(p.tokens) * units;
  const int pairs = kVec == 1 ? 1 : halves ? kVec : kVec / 2;   // of a unit: cosines of a thread
  int groups = p.heads;
  for (int per_thread = 2; per_thread <= kRopeMostHeads; ++per_thread) {
    const int g = (p.heads + per_thread - 1) / per_thread;
    if (one * g * (pairs > 4 ? 4 : 1) >= kRopeFill) groups = g;
  }
  const int64_t per_token = static_cast<int64_t>(units) * groups;
  int64_t tokens = per_token < kRopeThreads ? kRopeThreads / per_token : 1;
  const int split = per_token > kRopeThreads ? static_cast<int>((per_token + kRopeThreads - 1) / kRopeThreads) : 1;
  const int rows = static_cast<int>(tokens) * groups;
  RopeLaunch a{p, static_cast<int32_t>(tokens), static_cast<uint32_t>(rows) * turn_units, static_cast<uint32_t>(rows) * units,
               Divider(turn_units), Divider(copies > 0 ? copies : 1), Divider(groups)};
  const dim3 blocks(static_cast<unsigned>((p.tokens + tokens - 1) / tokens), split < 65535 ? split : 65535);
  auto launch = [&](auto kernel) { return launch_dependent(kernel, blocks, kRopeThreads, 0, stream, a); };
  // a head for each thread: no registers for more (42,129 tokens of one head, 96 of
  // 192, f16, out of place: 12.7 us with those of four heads, 10.5 so; a decode step
  // of 128 x 20 1.71 and 1.67)
  if (groups == p.heads)
    return halves ? launch(mla_rope_kernel<T, kVec, true, 1>) : launch(mla_rope_kernel<T, kVec, false, 1>);
  return halves ? launch(mla_rope_kernel<T, kVec, true, kRopeHeads>) : launch(mla_rope_kernel<T, kVec, false, kRopeHeads>);
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
