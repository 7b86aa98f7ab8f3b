// The rotary angle of a position.
//
// A pair turns by pos * turns * 2^-64 of a full turn, turns a 64-bit integer
// made on the host.  The wrapping product is that angle modulo a full turn,
// exactly, so positions of 2^31 lose as little as position 1.  Its upper 32
// bits split into the nearest quarter turn and a rest of at most an eighth, on
// which the Taylor polynomials of sine (to x^9) and cosine (to x^8) are exact
// to 2^-25; the rest enters them with 24 significant bits.  Two integer
// multiplies and shifts stand where a double-precision product and a range
// reduction would.
#pragma once

#include <cstdint>

namespace mla {

__device__ __forceinline__ void turn_cos_sin(uint64_t turns, int32_t pos, float* c, float* s) {
  const uint64_t phase = turns * static_cast<uint64_t>(static_cast<uint32_t>(pos));
  const uint32_t turn = static_cast<uint32_t>(phase >> 32);
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const int32_t rest = static_cast<int32_t>(turn - (quarter << 30));   // 2^-32 turns
  const float x = static_cast<float>(rest) * 1.4629180792671596e-9f;   // 2 pi 2^-32
  const float q = x * x;
  float a = fmaf(q, 1.f / 362880.f, -1.f / 5040.f);
  a = fmaf(a, q, 1.f / 120.f);
  a = fmaf(a, q, -1.f / 6.f);
  const float sn = fmaf(a * q, x, x);
  float b = fmaf(q, 1.f / 40320.f, -1.f / 720.f);
  b = fmaf(b, q, 1.f / 24.f);
  b = fmaf(b, q, -0.5f);
  const float cn = fmaf(b, q, 1.f);
  // quarter turns: (c, s), (-s, c), (-c, -s), (s, -c)
  const float u = quarter & 1u ? sn : cn, v = quarter & 1u ? cn : sn;
  *c = __uint_as_float(__float_as_uint(u) ^ ((quarter + 1u & 2u) << 30));
  *s = __uint_as_float(__float_as_uint(v) ^ ((quarter & 2u) << 30));
}

}  // namespace mla
