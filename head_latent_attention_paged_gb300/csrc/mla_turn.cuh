// The rotary angle of a position.
//
// A pair turns by pos * turns * 2^-64 of a full turn, turns a 64-bit integer
// made on the host.  The wrapping product is that angle modulo a full turn,
// exactly, so positions of 2^31 lose as little as position 1; its upper 32
// bits, read as a signed number of 2^-31 half turns, are the angle in [-pi,
// pi) to 2^-32 turns.  Two integer multiplies stand where a double-precision
// product and range reduction would.
#pragma once

#include <cstdint>

namespace mla {

__device__ __forceinline__ void turn_cos_sin(uint64_t turns, int32_t pos, float* c, float* s) {
  const uint64_t phase = turns * static_cast<uint64_t>(static_cast<uint32_t>(pos));
  const float half_turns =
      static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;   // 2^-31
  sincospif(half_turns, s, c);
}

}  // namespace mla
