// rotary_turn.h -- the coefficients of a rotary position.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace flare {

// What is left of position * freq, in turns, between -1/2 and 1/2.
__device__ __forceinline__ double turn_fraction(int32_t position, double freq) {
  const double turns = (double)position * (freq * 0.15915494309189533577);
  return turns - rint(turns);
}

// m cos and m sin of position * freq (sign: -1 for the reverse mode).
__device__ __forceinline__ float2 turn(int32_t position, double freq, float m, float sign) {
  float s, c;
  sincospif(2.0f * (float)turn_fraction(position, freq), &s, &c);
  return make_float2(m * c, m * sign * s);
}

}  // namespace flare
