// fp4.h -- the 4-bit values of a cache: groups of 32 channels, each value one of 0,
// 1/2, 1, 3/2, 2, 3, 4, 6 with a sign (codes 0..7, 8 the sign) times 2^(byte - 127).
#pragma once

#include "device_common.h"

namespace flare {

constexpr int kFp4Group = 32;  // channels that share a scale

// What of a double decides its code and its group's scale, borders of few bits: the upper
// half, its last bit set where the lower one is not zero.
struct Upper {
  uint32_t w;
};
__device__ __forceinline__ Upper upper(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  return {(uint32_t)(b >> 32) | ((uint32_t)b != 0 ? 1u : 0u)};
}

// The magnitude's bits, ordered as the magnitudes are, NaN above all.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t abs_bits(Upper x) { return x.w & 0x7fffffffu; }

// The scale of a group whose largest magnitude has these bits: its exponent less two
// (the largest code is 6 = 1.5 2^2), and one more where the largest value is above 7
// units: 7 is cut to 6, as far as half a step there, and more would be cut further.  1 to
// 252, so that every value is a normal finite bf16 or the subnormal it would be; 255: the
// group holds an infinity or NaN, and is NaN.
template <typename T> __device__ __forceinline__ int fp4_scale(uint32_t top) {
  constexpr int kMantissa = __is_same(T, Upper) ? 20 : 23, kBias = __is_same(T, Upper) ? 1023 : 127;
  if (top >= (uint32_t)(2 * kBias + 1) << kMantissa) return 255;
  const int e = (int)(top >> kMantissa) - kBias + 127 - 2 + ((top & ((1u << kMantissa) - 1)) > 3u << (kMantissa - 2));
  return e < 1 ? 1 : e > 252 ? 252 : e;
}

// x / 2^(byte - 127) as a float whose rounding to a code is x's: exact, or with as many bits
// as a border's and a last one that keeps it off the border.
__device__ __forceinline__ float fp4_units(float x, int byte) { return x * __uint_as_float((uint32_t)(254 - byte) << 23); }
__device__ __forceinline__ float fp4_units(Upper x, int byte) {
  // the exponent's bias changed, below 2^-127 to 0 and beyond 2^80 to that
  const int v = (int)(x.w & 0x7fffffffu) - ((1023 - 254 + byte) << 20), top = 207 << 20;
  return __uint_as_float((uint32_t)(v < 0 ? 0 : v > top ? top : v) << 3 | (x.w & 0x80000000u));
}

// The codes of eight channels, halfway to the even code, beyond 6 to 6.
template <typename T> __device__ __forceinline__ uint32_t fp4_codes(const T (&x)[8], int byte) {
  if (byte == 255) return 0;
  float z[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = fp4_units(x[e], byte);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, z[0], z[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, z[2], z[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, z[4], z[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, z[6], z[7], 1.0f, 3);
}

// The bf16 values of the codes in byte SEL of w, the lower four bits first: the
// instruction takes the scale from the exponent's bits alone (255: NaN).
template <int SEL> __device__ __forceinline__ uint32_t fp4_pair(uint32_t w, uint32_t scale_bits) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, __uint_as_float(scale_bits), SEL));
}

}  // namespace flare
