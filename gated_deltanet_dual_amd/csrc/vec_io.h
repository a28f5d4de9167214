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

template <typename IO, int VEC, bool TAIL>
__device__ __forceinline__ void load_vec(const IO *p, int n, float *f) {
  if (!TAIL || n >= VEC) {
    Vec<IO, VEC>::load(p, f);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = e < n ? io_traits<IO>::to_f(p[e]) : 0.0f;
  }
}
template <typename IO, int VEC, bool TAIL>
__device__ __forceinline__ void store_vec(IO *p, int n, const float *f) {
  if (!TAIL || n >= VEC) {
    Vec<IO, VEC>::store(p, f);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < n) p[e] = io_traits<IO>::from_f(f[e]);
  }
}

}  // namespace flare
