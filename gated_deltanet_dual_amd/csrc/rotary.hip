// rotary.hip -- rotary positions on q and k, and the serving form that writes
// the turned keys and the values into the paged cache.
//
//   (a, b) -> m (a cos - b sin, a sin + b cos),  angle = position * freq
//
// for the pairs (i, half + i) or (2i, 2i + 1) of a head's first 2 half
// channels; the others pass through.  The reverse mode turns by the negative
// angle.  position * freq in turns is formed and reduced in 64 bits: in 32 an
// angle at position 10^6 is off by 0.06 rad.  The product is off by some 2^-52 of
// itself, 2^-32 turns at position 2^20; sine and cosine of what is left are fp32's.
#include <hip/hip_runtime.h>

#include "fast_div.h"
#include "layer_launch.h"
#include "vec_io.h"

namespace flare {
namespace {

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
// Memory bounds it: 32768 tokens, 16 + 4 heads of 128, 32 of them turned, bf16: 336 MB
// in 64 to 66 us, 5.2 TB/s (two tokens a workgroup).  The serving form over 1024 tokens
// takes 5.2 us where a launch takes 3.7: positions and frequencies, the slot, and the row
// itself are three latencies in a row, and in the interleaved layout 71 % of the cycles of
// the coefficients' LDS reads are bank conflicts.
template <typename IO, int VEC, bool TAIL>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, RotaryPlan p) {
  extern __shared__ float2 coef[];  // [tb][half]
  const int64_t t0 = (int64_t)blockIdx.x * p.tb;
  const int n = (int)(a.tokens - t0 < p.tb ? a.tokens - t0 : p.tb);
  for (int i = threadIdx.x; i < n * a.half; i += blockDim.x) {
    const int t = fast_div(i, p.half), j = i - t * a.half;
    coef[i] = turn(a.positions[t0 + t], a.freqs[j], a.mscale, a.sign);
  }
  __syncthreads();
  const auto [per, v_per, items] = rotary_items(a, VEC);
  const int turned = rotary_turned_items(a, VEC), heads = a.q_heads + a.k_heads;
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
    // the item's two places in the row and how many channels it has there (n1 <= 0: none)
    const bool copy = kind == 2 || j >= turned;
    int c0, c1, n0, n1;
    if (copy) {
      c0 = (kind == 2 ? 0 : 2 * a.half) + 2 * (kind == 2 ? j : j - turned) * VEC;
      c1 = c0 + VEC;
      n0 = a.dim - c0;
      n1 = a.dim - c1;
    } else if (!a.interleaved) {
      c0 = j * VEC;
      c1 = a.half + c0;
      n0 = n1 = a.half - c0;
    } else {
      c0 = 2 * j * VEC;
      c1 = c0 + VEC;
      n0 = 2 * a.half - c0;
      n1 = 2 * a.half - c1;
    }
    if (n1 <= 0) c1 = c0;  // read what is there, write it once
    const int m1 = n1 <= 0 ? n0 : n1;
    float x[VEC], y[VEC];
    load_vec<IO, VEC, TAIL>(src + c0, n0, x);
    load_vec<IO, VEC, TAIL>(src + c1, m1, y);
    if (!copy) {
      if (!a.interleaved) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float2 w = cf[TAIL && e >= n0 ? c0 : c0 + e];
          const float u = x[e], v = y[e];
          x[e] = u * w.x - v * w.y;
          y[e] = u * w.y + v * w.x;
        }
      } else {
        const float2 *cx = cf + c0 / 2, *cy = cf + c1 / 2;
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const float2 w = cx[TAIL && e >= n0 ? 0 : e / 2], z = cy[TAIL && e >= m1 ? 0 : e / 2];
          const float u = x[e], v = x[e + 1], s = y[e], t2 = y[e + 1];
          x[e] = u * w.x - v * w.y;
          x[e + 1] = u * w.y + v * w.x;
          y[e] = s * z.x - t2 * z.y;
          y[e + 1] = s * z.y + t2 * z.x;
        }
      }
    }
    store_vec<IO, VEC, TAIL>(dst + c0, n0, x);
    if (n1 > 0) store_vec<IO, VEC, TAIL>(dst + c1, n1, y);
  }
}

}  // namespace

template <typename IO, int VEC>
static void launch(const RotaryArgs &a, hipStream_t st) {
  const bool tail = (a.interleaved ? 2 * a.half : a.half) % VEC != 0 || (a.dim - 2 * a.half) % VEC != 0 ||
                    (a.slots && a.dim % VEC != 0);
  const RotaryItems it = rotary_items(a, VEC);
  RotaryPlan p;
  p.tb = rotary_block_tokens(a);
  p.half = make_fast_div(a.half > 0 ? a.half : 1);
  p.items = make_fast_div(it.token);
  p.per = make_fast_div(it.per);
  p.v_per = make_fast_div(it.v_per > 0 ? it.v_per : 1);
  const int grid = (int)((a.tokens + p.tb - 1) / p.tb);
  const size_t lds = (size_t)p.tb * (a.half > 0 ? a.half : 1) * sizeof(float2);
  if (tail) rotary_kernel<IO, VEC, true><<<grid, 256, lds, st>>>(a, p);
  else rotary_kernel<IO, VEC, false><<<grid, 256, lds, st>>>(a, p);
}

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  TimedLaunch tl(K_ROTARY, st);
  if (a.bf16) launch<u16, rotary_vec(true)>(a, st);
  else launch<float, rotary_vec(false)>(a, st);
  return hipGetLastError();
}

}  // namespace flare
