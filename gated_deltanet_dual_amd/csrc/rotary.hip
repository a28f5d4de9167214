// rotary.hip -- rotary positions on q and k, and the serving form that writes
// the turned keys and the values into the paged cache.
//
//   (a, b) -> m (a cos - b sin, a sin + b cos),  angle = position * freq
//
// for the pairs (i, half + i) or (2i, 2i + 1) of a head's first 2 half
// channels; the others pass through.  The reverse mode turns by the negative
// angle.  position * freq in turns is formed and reduced in 64 bits: in 32 an
// angle at position 10^6 is off by 0.06 rad.
#include <hip/hip_runtime.h>

#include "device_common.h"
#include "fast_div.h"
#include "layer_launch.h"

namespace flare {
namespace {

template <typename IO, int VEC> struct Pack;
template <> struct Pack<u16, 8> {
  float f[8];
  __device__ __forceinline__ void load(const u16 *p) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(w[e] << 16);
      f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void store(u16 *p) const {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                               pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};
template <> struct Pack<float, 4> {
  float f[4];
  __device__ __forceinline__ void load(const float *p) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  }
  __device__ __forceinline__ void store(float *p) const {
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <typename IO> struct Pack<IO, 1> {
  float f[1];
  __device__ __forceinline__ void load(const IO *p) { f[0] = io_traits<IO>::to_f(*p); }
  __device__ __forceinline__ void store(IO *p) const { *p = io_traits<IO>::from_f(f[0]); }
};

// m cos and m sin of position * freq (sign: -1 for the reverse mode).
__device__ __forceinline__ float2 turn(int32_t position, double freq, float m, float sign) {
  const double turns = (double)position * (freq * 0.15915494309189533577);
  float s, c;
  sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
  return make_float2(m * c, m * sign * s);
}

struct RotaryPlan {
  int tb;                            // tokens a workgroup
  FastDiv half, items, per, v_per;   // by half, a token's, a head's and a value head's work items
};

// One workgroup: `tb` tokens.  Their coefficients first, to LDS, so that a
// token's angles are formed once for all its heads; then the heads' vectors.
// A head's work items hold two vectors each, so that a thread has two loads in
// flight.  First those that turn: a vector of each half (of a pair's two elements
// where vec is 1), or in the interleaved layout two whole vectors; then copies.  A
// count that is odd leaves the last item one vector.
__host__ __device__ inline int turned_items(const RotaryArgs &a, int vec) {
  return a.interleaved && vec > 1 ? (2 * a.half / vec + 1) / 2 : a.half / vec;
}
__host__ __device__ inline int copy_items(int channels, int vec) { return (channels / vec + 1) / 2; }

template <typename IO, int VEC>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, RotaryPlan p) {
  extern __shared__ float2 coef[];  // [tb][half]
  const int64_t t0 = (int64_t)blockIdx.x * p.tb;
  const int n = (int)(a.tokens - t0 < p.tb ? a.tokens - t0 : p.tb);
  for (int i = threadIdx.x; i < n * a.half; i += blockDim.x) {
    const int t = fast_div(i, p.half), j = i - t * a.half;
    coef[i] = turn(a.positions[t0 + t], a.freqs[j], a.mscale, a.sign);
  }
  __syncthreads();
  const int turned = turned_items(a, VEC), per = turned + copy_items(a.dim - 2 * a.half, VEC);
  const int heads = a.q_heads + a.k_heads;
  const int v_per = a.slots ? copy_items(a.dim, VEC) : 0;
  const int items = heads * per + a.k_heads * v_per;
  const int64_t cache_tokens = a.num_pages * a.page;
  for (int i = threadIdx.x; i < n * items; i += blockDim.x) {
    const int t = fast_div(i, p.items), r = i - t * items;
    const int64_t tok = t0 + t;
    int head, j, kind;  // kind 0 q, 1 k, 2 v
    if (r < heads * per) {
      head = fast_div(r, p.per);
      j = r - head * per;
      kind = head >= a.q_heads;
      if (kind) head -= a.q_heads;
    } else {
      const int rv = r - heads * per;
      head = fast_div(rv, p.v_per);
      j = rv - head * v_per;
      kind = 2;
    }
    const IO *src;
    IO *dst;
    if (kind == 0) {
      src = (const IO *)a.q + tok * a.q_stride + (int64_t)head * a.dim;
      dst = (IO *)a.q_out + (tok * a.q_heads + head) * a.dim;
    } else {
      src = kind == 1 ? (const IO *)a.k + tok * a.k_stride + (int64_t)head * a.dim
                      : (const IO *)a.v + tok * a.v_stride + (int64_t)head * a.dim;
      if (a.slots) {
        const int64_t slot = a.slots[tok];
        if (slot < 0 || slot >= cache_tokens) continue;
        const int64_t pg = slot / a.page;
        dst = (kind == 1 ? (IO *)a.k_cache : (IO *)a.v_cache) +
              ((pg * a.k_heads + head) * a.page + (slot - pg * a.page)) * a.dim;
      } else {
        dst = (IO *)a.k_out + (tok * a.k_heads + head) * a.dim;
      }
    }
    const float2 *cf = coef + t * a.half;
    // the item's two places in the row; c1 < 0: it has one
    const bool copy = kind == 2 || j >= turned;
    int c0, c1;
    if (copy) {
      const int first = kind == 2 ? 0 : 2 * a.half, vecs = (a.dim - first) / VEC;
      c0 = first + 2 * (kind == 2 ? j : j - turned) * VEC;
      c1 = c0 + VEC < first + vecs * VEC ? c0 + VEC : -1;
    } else if (!a.interleaved) {
      c0 = j * VEC;
      c1 = a.half + c0;
    } else if (VEC == 1) {
      c0 = 2 * j;
      c1 = c0 + 1;
    } else {
      c0 = 2 * j * VEC;
      c1 = c0 + VEC < 2 * a.half ? c0 + VEC : -1;
    }
    Pack<IO, VEC> x, y;
    x.load(src + c0);
    y.load(src + (c1 < 0 ? c0 : c1));
    if (!copy) {
      if (!a.interleaved || VEC == 1) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float2 w = cf[j * VEC + e];
          const float u = x.f[e], v = y.f[e];
          x.f[e] = u * w.x - v * w.y;
          y.f[e] = u * w.y + v * w.x;
        }
      } else {
        const float2 *cx = cf + c0 / 2, *cy = cf + (c1 < 0 ? c0 : c1) / 2;
#pragma unroll
        for (int e = 0; e + 1 < VEC; e += 2) {
          const float2 w = cx[e / 2], z = cy[e / 2];
          const float u = x.f[e], v = x.f[e + 1], s = y.f[e], t2 = y.f[e + 1];
          x.f[e] = u * w.x - v * w.y;
          x.f[e + 1] = u * w.y + v * w.x;
          y.f[e] = s * z.x - t2 * z.y;
          y.f[e + 1] = s * z.y + t2 * z.x;
        }
      }
    }
    x.store(dst + c0);
    if (c1 >= 0) y.store(dst + c1);
  }
}

bool vec_ok(const void *p, int64_t stride, int elem) { return ((uintptr_t)p & 15) == 0 && (stride * elem) % 16 == 0; }

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  const int e = a.bf16 ? 2 : 4, vec = 16 / e;
  bool wide = a.dim % vec == 0 && (a.interleaved ? 2 * a.half : a.half) % vec == 0 && vec_ok(a.q, a.q_stride, e) &&
              vec_ok(a.q_out, a.dim, e);
  if (a.k_heads > 0) {
    wide = wide && vec_ok(a.k, a.k_stride, e);
    if (a.slots)
      wide = wide && vec_ok(a.v, a.v_stride, e) && vec_ok(a.k_cache, a.dim, e) && vec_ok(a.v_cache, a.dim, e);
    else
      wide = wide && vec_ok(a.k_out, a.dim, e);
  }
  RotaryPlan p;
  p.tb = 1;
  while (p.tb < 8 && a.tokens / (2 * p.tb) >= 4096 && 2 * p.tb * a.half <= 2048) p.tb *= 2;
  const int v = wide ? vec : 1, per = turned_items(a, v) + copy_items(a.dim - 2 * a.half, v);
  const int v_per = a.slots ? copy_items(a.dim, v) : 0;
  const int items = (a.q_heads + a.k_heads) * per + a.k_heads * v_per;
  p.half = make_fast_div(a.half > 0 ? a.half : 1);
  p.items = make_fast_div(items);
  p.per = make_fast_div(per);
  p.v_per = make_fast_div(v_per > 0 ? v_per : 1);
  const int grid = (int)((a.tokens + p.tb - 1) / p.tb);
  const size_t lds = (size_t)p.tb * (a.half > 0 ? a.half : 1) * sizeof(float2);
  TimedLaunch tl(K_ROTARY, st);
  if (a.bf16) {
    if (wide) rotary_kernel<u16, 8><<<grid, 256, lds, st>>>(a, p);
    else rotary_kernel<u16, 1><<<grid, 256, lds, st>>>(a, p);
  } else {
    if (wide) rotary_kernel<float, 4><<<grid, 256, lds, st>>>(a, p);
    else rotary_kernel<float, 1><<<grid, 256, lds, st>>>(a, p);
  }
  return hipGetLastError();
}

}  // namespace flare
