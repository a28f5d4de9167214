// vec_io.h -- rows moved 16 bytes at a time whatever their alignment and width.
#pragma once

#include "device_common.h"

namespace flare {

// VEC consecutive elements of a row as fp32.  The GPU loads and stores 16 bytes at
// any byte address (an access across a line costs one more), so a row of odd width
// or start goes the same way; only a row's last vector can be short: `n` of its
// elements exist, the others are zeros.  TAIL: whether short vectors occur.
template <typename IO, int VEC> struct Vec;
template <> struct Vec<u16, 8> {
  static __device__ __forceinline__ void load(const u16 *p, float *f) {
    uint4 v;
    __builtin_memcpy(&v, p, 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(w[e] << 16);
      f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(u16 *p, const float *f) {
    const uint4 v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                               pack_bf16x2(f[6], f[7]));
    __builtin_memcpy(p, &v, 16);
  }
};
template <> struct Vec<float, 4> {
  static __device__ __forceinline__ void load(const float *p, float *f) { __builtin_memcpy(f, p, 16); }
  static __device__ __forceinline__ void store(float *p, const float *f) { __builtin_memcpy(p, f, 16); }
};
template <> struct Vec<float, 8> {
  static __device__ __forceinline__ void load(const float *p, float *f) {
    Vec<float, 4>::load(p, f);
    Vec<float, 4>::load(p + 4, f + 4);
  }
  static __device__ __forceinline__ void store(float *p, const float *f) {
    Vec<float, 4>::store(p, f);
    Vec<float, 4>::store(p + 4, f + 4);
  }
};

// A short vector goes as its count's powers of two: 4, 2 and 1 elements, each there
// or not, in place of one access an element.
template <typename IO, int VEC>
__device__ __forceinline__ void load_short(const IO *p, int n, float *f) {
  IO four[4] = {}, two[2] = {}, one[1] = {};
  if (VEC > 4 && (n & 4)) __builtin_memcpy(four, p, 4 * sizeof(IO));
  if (n & 2) __builtin_memcpy(two, p + (n & (VEC - 4)), 2 * sizeof(IO));
  if (n & 1) __builtin_memcpy(one, p + (n & (VEC - 2)), sizeof(IO));
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    // element e is the one if it is the last of an odd count, else in the four below 4 where there are four, else in the two
    const float a = VEC > 4 && e < 4 ? io_traits<IO>::to_f(four[e & 3]) : 0.0f;
    const float b = io_traits<IO>::to_f(two[e & 1]);
    const float c = io_traits<IO>::to_f(one[0]);
    const bool in_four = VEC > 4 && e < 4 && (n & 4);
    const bool in_one = (n & 1) && e == n - 1;
    f[e] = e >= n ? 0.0f : in_one ? c : in_four ? a : b;
  }
}
template <typename IO, int VEC>
__device__ __forceinline__ void store_short(IO *p, int n, const float *f) {
  IO x[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] = io_traits<IO>::from_f(f[e]);
  const bool four = VEC > 4 && (n & 4);
  if (four) __builtin_memcpy(p, x, 4 * sizeof(IO));
  if (n & 2) {
    const IO two[2] = {four ? x[VEC > 4 ? 4 : 0] : x[0], four ? x[VEC > 4 ? 5 : 1] : x[1]};
    __builtin_memcpy(p + (n & (VEC - 4)), two, 2 * sizeof(IO));
  }
  if (n & 1) {
    IO one = x[0];
#pragma unroll
    for (int e = 2; e < VEC; e += 2)
      if (n == e + 1) one = x[e];
    p[n - 1] = one;
  }
}

template <typename IO, int VEC, bool TAIL>
__device__ __forceinline__ void load_vec(const IO *p, int n, float *f) {
  if (!TAIL || n >= VEC) Vec<IO, VEC>::load(p, f);
  else load_short<IO, VEC>(p, n, f);
}
template <typename IO, int VEC, bool TAIL>
__device__ __forceinline__ void store_vec(IO *p, int n, const float *f) {
  if (!TAIL || n >= VEC) Vec<IO, VEC>::store(p, f);
  else store_short<IO, VEC>(p, n, f);
}

}  // namespace flare
