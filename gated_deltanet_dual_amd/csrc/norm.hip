// norm.hip -- the norms before and after a block, fused with its gate and
// residual scale, forward and reverse mode.
//
//   gated norm     y = x r w act(g),  r = 1 / sqrt(mean x^2 + eps), per head row
//   residual norm  n = x r1 w1 (or x);  h = res + s act(g) n;  y = h r2 w2
//
// Reverse of a normalised row u = x r with incoming gradient du:
//   dx = r (du - u mean(du u)).
#include <hip/hip_runtime.h>

#include "device_common.h"
#include "layer_launch.h"

namespace flare {
namespace {

// VEC consecutive elements of a row, as fp32.
template <typename IO, int VEC> struct Vec;
template <> struct Vec<u16, 8> {
  static __device__ __forceinline__ void load(const u16 *p, float *f) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(w[e] << 16);
      f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(u16 *p, const float *f) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                               pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};
template <> struct Vec<float, 4> {
  static __device__ __forceinline__ void load(const float *p, float *f) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  }
  static __device__ __forceinline__ void store(float *p, const float *f) {
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
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
template <typename IO> struct Vec<IO, 1> {
  static __device__ __forceinline__ void load(const IO *p, float *f) { f[0] = io_traits<IO>::to_f(*p); }
  static __device__ __forceinline__ void store(IO *p, const float *f) { *p = io_traits<IO>::from_f(f[0]); }
};

__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// f = act(g) of a vector's elements (1 without a gate, act < 0).  The choice is
// made once for the vector: inside the element loop it would cut the code at
// every element.
template <int VEC> __device__ __forceinline__ void gate_values(const float *g, int act, float *f) {
  if (act == FLARE_GATE_SILU) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = g[e] * sigmoid(g[e]);
  } else if (act == FLARE_GATE_SIGMOID) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = sigmoid(g[e]);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = act == FLARE_GATE_LINEAR ? g[e] : 1.0f;
  }
}
// and the derivative d (0 without a gate)
template <int VEC> __device__ __forceinline__ void gate_values_d(const float *g, int act, float *f, float *d) {
  if (act == FLARE_GATE_SILU) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float x = g[e], p = sigmoid(x);  // f may be g
      f[e] = x * p;
      d[e] = p * (1.0f + x * (1.0f - p));
    }
  } else if (act == FLARE_GATE_SIGMOID) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      f[e] = sigmoid(g[e]);
      d[e] = f[e] * (1.0f - f[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      f[e] = act == FLARE_GATE_LINEAR ? g[e] : 1.0f;
      d[e] = act == FLARE_GATE_LINEAR ? 1.0f : 0.0f;
    }
  }
}
// The vector c of an fp32 weight, or ones where it is absent.
template <int VEC> __device__ __forceinline__ void load_or_one(const float *w, int c, float *f) {
  if (w) {
    Vec<float, VEC>::load(w + c * VEC, f);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = 1.0f;
  }
}

// A row is held by a team of `team` threads, a power of two: up to a wave
// (several teams to a wave, sums by lane exchanges) or a whole workgroup
// (BLOCK: sums through LDS).  Thread i of the team holds the vectors i,
// i + team, ... of the row in registers, so every input is read once.
template <bool BLOCK> struct Team {
  int size, lane;
  __device__ __forceinline__ float sum(float x, float *red) const {
    if constexpr (!BLOCK) {
      for (int o = size >> 1; o > 0; o >>= 1) x += __shfl_xor(x, o);
      return x;
    } else {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
      const int w = threadIdx.x >> 6, nw = size >> 6;
      __syncthreads();  // the previous sum's reads of red
      if ((threadIdx.x & 63) == 0) red[w] = x;
      __syncthreads();
      float s = 0.0f;
      for (int i = 0; i < nw; ++i) s += red[i];
      return s;
    }
  }
};

// ---------------------------------------------------------------- gated norm
template <typename IO, int VEC, int NV, bool BLOCK, int THREADS>
__global__ __launch_bounds__(THREADS) void gated_norm_kernel(GatedNormArgs a, int team) {
  __shared__ float red[16];
  const Team<BLOCK> tm{team, BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (team - 1))};
  const int per = BLOCK ? 1 : blockDim.x / team;
  const uint32_t rows = (uint32_t)(a.tokens * a.heads);
  const int nv = a.dim / VEC;
  for (uint32_t row = blockIdx.x * per + (BLOCK ? 0 : threadIdx.x / team); row < rows; row += gridDim.x * per) {
    const uint32_t t = row / (uint32_t)a.heads, h = row - t * (uint32_t)a.heads;
    const IO *x = (const IO *)a.x + (int64_t)t * a.x_stride + (int64_t)h * a.dim;
    const IO *g = (const IO *)a.gate + (int64_t)t * a.gate_stride + (int64_t)h * a.dim;
    float xv[NV][VEC], gv[NV][VEC], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        Vec<IO, VEC>::load(x + c * VEC, xv[i]);
        if (a.act >= 0) Vec<IO, VEC>::load(g + c * VEC, gv[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss += xv[i][e] * xv[i][e];
      }
    }
    ss = tm.sum(ss, red);
    const float r = 1.0f / sqrtf(ss / (float)a.dim + a.eps);
    if (a.rstd && tm.lane == 0) a.rstd[row] = r;
    IO *y = (IO *)a.y + (int64_t)row * a.dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        float w[VEC], o[VEC];
        Vec<float, VEC>::load(a.weight + c * VEC, w);
        gate_values<VEC>(gv[i], a.act, o);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] *= xv[i][e] * r * w[e];
        Vec<IO, VEC>::store(y + c * VEC, o);
      }
    }
  }
}

// Adds the threads' column sums of a workgroup: `acc` of every team for the
// vectors it holds, into part[blockIdx.x][dim].
template <int VEC, int NV, bool BLOCK>
__device__ __forceinline__ void write_partial(const float (&acc)[NV][VEC], const Team<BLOCK> &tm, int dim, float *part,
                                              float *lds) {
  const int nv = dim / VEC;
  float *out = part + (int64_t)blockIdx.x * dim;
  if constexpr (BLOCK) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * tm.size;
      if (c < nv) Vec<float, VEC>::store(out + c * VEC, acc[i]);
    }
  } else {
    // lds [blockDim.x][VEC]: one vector of every thread at a time
    const int teams = blockDim.x / tm.size;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e) lds[threadIdx.x * VEC + e] = acc[i][e];
      __syncthreads();
      for (int j = threadIdx.x; j < tm.size * VEC; j += blockDim.x) {
        const int c = i * tm.size * VEC + j;
        if (c < nv * VEC) {
          float s = 0.0f;
          for (int k = 0; k < teams; ++k) s += lds[k * tm.size * VEC + j];
          out[c] = s;
        }
      }
    }
  }
}

template <typename IO, int VEC, int NV, bool BLOCK, int THREADS>
__global__ __launch_bounds__(THREADS) void gated_norm_bwd_kernel(GatedNormArgs a, int team) {
  __shared__ float red[16];
  __shared__ float cols[BLOCK ? 1 : 256 * VEC];
  const Team<BLOCK> tm{team, BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (team - 1))};
  const int per = BLOCK ? 1 : blockDim.x / team;
  const uint32_t rows = (uint32_t)(a.tokens * a.heads);
  const int nv = a.dim / VEC;
  float dw[NV][VEC] = {};
  float w[NV][VEC] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (tm.lane + i * team < nv) Vec<float, VEC>::load(a.weight + (tm.lane + i * team) * VEC, w[i]);
  for (uint32_t row = blockIdx.x * per + (BLOCK ? 0 : threadIdx.x / team); row < rows; row += gridDim.x * per) {
    const uint32_t t = row / (uint32_t)a.heads, h = row - t * (uint32_t)a.heads;
    const int64_t hd = (int64_t)h * a.dim;
    const IO *x = (const IO *)a.x + (int64_t)t * a.x_stride + hd;
    const IO *g = (const IO *)a.gate + (int64_t)t * a.gate_stride + hd;
    const IO *dy = (const IO *)a.dy + (int64_t)t * a.dy_stride + hd;
    const float r = a.rstd[row];
    float u[NV][VEC], du[NV][VEC], gv[NV][VEC], dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        Vec<IO, VEC>::load(x + c * VEC, u[i]);
        Vec<IO, VEC>::load(dy + c * VEC, du[i]);
        if (a.act >= 0) Vec<IO, VEC>::load(g + c * VEC, gv[i]);
        float f[VEC], d[VEC];
        gate_values_d<VEC>(gv[i], a.act, f, d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          u[i][e] *= r;
          const float du_u = du[i][e] * u[i][e];
          dw[i][e] += du_u * f[e];
          gv[i][e] = du_u * w[i][e] * d[e];
          du[i][e] *= w[i][e] * f[e];
          dot += du[i][e] * u[i][e];
        }
      }
    }
    dot = tm.sum(dot, red) / (float)a.dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = r * (du[i][e] - u[i][e] * dot);
        Vec<IO, VEC>::store((IO *)a.dx + (int64_t)row * a.dim + c * VEC, o);
        if (a.act >= 0) Vec<IO, VEC>::store((IO *)a.dgate + (int64_t)row * a.dim + c * VEC, gv[i]);
      }
    }
  }
  write_partial<VEC, NV, BLOCK>(dw, tm, a.dim, a.part, cols);
}

// ---------------------------------------------------------------- residual norm
template <typename IO, typename RES, int VEC, int NV, bool BLOCK, int THREADS>
__global__ __launch_bounds__(THREADS) void residual_norm_kernel(ResidualNormArgs a, int team) {
  __shared__ float red[16];
  const Team<BLOCK> tm{team, BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (team - 1))};
  const int per = BLOCK ? 1 : blockDim.x / team;
  const int nv = a.dim / VEC;
  for (int64_t row = (int64_t)blockIdx.x * per + (BLOCK ? 0 : threadIdx.x / team); row < a.tokens;
       row += (int64_t)gridDim.x * per) {
    const IO *x = (const IO *)a.x + row * a.x_stride;
    const IO *g = (const IO *)a.gate + row * a.gate_stride;
    const RES *res = (const RES *)a.residual + row * a.dim;
    float xv[NV][VEC], gv[NV][VEC], hv[NV][VEC], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        Vec<IO, VEC>::load(x + c * VEC, xv[i]);
        Vec<RES, VEC>::load(res + c * VEC, hv[i]);
        if (a.act >= 0) Vec<IO, VEC>::load(g + c * VEC, gv[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss += xv[i][e] * xv[i][e];
      }
    }
    float r1 = 1.0f;
    if (a.w_post) r1 = 1.0f / sqrtf(tm.sum(ss, red) / (float)a.dim + a.eps);
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        float w1[VEC], sc[VEC], f[VEC];
        load_or_one<VEC>(a.w_post, c, w1);
        load_or_one<VEC>(a.scale, c, sc);
        gate_values<VEC>(gv[i], a.act, f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          hv[i][e] += xv[i][e] * r1 * w1[e] * f[e] * sc[e];
          ss += hv[i][e] * hv[i][e];
        }
        Vec<RES, VEC>::store((RES *)a.h + row * a.dim + c * VEC, hv[i]);
      }
    }
    // the second norm is of h before h's own rounding
    const float r2 = 1.0f / sqrtf(tm.sum(ss, red) / (float)a.dim + a.eps);
    if (a.rstd && tm.lane == 0) {
      a.rstd[2 * row] = r1;
      a.rstd[2 * row + 1] = r2;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        float w2[VEC], o[VEC];
        Vec<float, VEC>::load(a.w_pre + c * VEC, w2);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = hv[i][e] * r2 * w2[e];
        Vec<IO, VEC>::store((IO *)a.y + row * a.dim + c * VEC, o);
      }
    }
  }
}

template <typename IO, typename RES, int VEC, int NV, bool BLOCK, int THREADS>
__global__ __launch_bounds__(THREADS) void residual_norm_bwd_kernel(ResidualNormArgs a, int team) {
  __shared__ float red[16];
  __shared__ float cols[BLOCK ? 1 : 256 * VEC];
  const Team<BLOCK> tm{team, BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (team - 1))};
  const int per = BLOCK ? 1 : blockDim.x / team;
  const int nv = a.dim / VEC;
  float dw2[NV][VEC] = {}, dw1[NV][VEC] = {}, ds[NV][VEC] = {};
  // the weights of a thread's one vector stay in registers over its rows (of 128
  // registers that larger workgroups leave, they would be 3 VEC too many)
  constexpr bool KEEP = NV == 1 && THREADS <= 256;
  float w2[VEC] = {}, w1[VEC] = {}, sc[VEC] = {};
  if (KEEP && tm.lane < nv) {
    Vec<float, VEC>::load(a.w_pre + tm.lane * VEC, w2);
    load_or_one<VEC>(a.w_post, tm.lane, w1);
    load_or_one<VEC>(a.scale, tm.lane, sc);
  }
  for (int64_t row = (int64_t)blockIdx.x * per + (BLOCK ? 0 : threadIdx.x / team); row < a.tokens;
       row += (int64_t)gridDim.x * per) {
    const IO *x = (const IO *)a.x + row * a.x_stride;
    const IO *g = (const IO *)a.gate + row * a.gate_stride;
    const RES *res = (const RES *)a.residual + row * a.dim;
    const float r1 = a.rstd[2 * row], r2 = a.rstd[2 * row + 1];
    // h again, in fp32 as the forward formed it
    float n[NV][VEC], f[NV][VEC], df[NV][VEC], u[NV][VEC], dy[NV][VEC], dh[NV][VEC], dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        Vec<IO, VEC>::load(x + c * VEC, n[i]);
        Vec<RES, VEC>::load(res + c * VEC, u[i]);
        Vec<IO, VEC>::load((const IO *)a.dy + row * a.dim + c * VEC, dy[i]);
        if (a.act >= 0) Vec<IO, VEC>::load(g + c * VEC, f[i]);
        if (a.dh) {
          Vec<RES, VEC>::load((const RES *)a.dh + row * a.dim + c * VEC, dh[i]);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) dh[i][e] = 0.0f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        if constexpr (!KEEP) {
          Vec<float, VEC>::load(a.w_pre + c * VEC, w2);
          load_or_one<VEC>(a.w_post, c, w1);
          load_or_one<VEC>(a.scale, c, sc);
        }
        gate_values_d<VEC>(f[i], a.act, f[i], df[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          n[i][e] *= r1;  // the normalised x (x itself without a post-norm: r1 is 1)
          u[i][e] = (u[i][e] + n[i][e] * w1[e] * f[i][e] * sc[e]) * r2;
          dw2[i][e] += dy[i][e] * u[i][e];
          dy[i][e] *= w2[e];
          dot += dy[i][e] * u[i][e];
        }
      }
    }
    dot = tm.sum(dot, red) / (float)a.dim;
    float dot1 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        if constexpr (!KEEP) {
          load_or_one<VEC>(a.w_post, c, w1);
          load_or_one<VEC>(a.scale, c, sc);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float d = dh[i][e] + r2 * (dy[i][e] - u[i][e] * dot);
          dh[i][e] = d;
          const float dz = d * n[i][e] * w1[e];  // z dh: what the gate and the scale see
          df[i][e] *= dz * sc[e];
          ds[i][e] += dz * f[i][e];
          const float t = d * sc[e] * f[i][e];  // the gradient of z
          dw1[i][e] += t * n[i][e];
          u[i][e] = t * w1[e];
          dot1 += u[i][e] * n[i][e];
        }
        Vec<RES, VEC>::store((RES *)a.dres + row * a.dim + c * VEC, dh[i]);
        if (a.act >= 0) Vec<IO, VEC>::store((IO *)a.dgate + row * a.dim + c * VEC, df[i]);
      }
    }
    // without a post-norm x's gradient is z's
    dot1 = a.w_post ? tm.sum(dot1, red) / (float)a.dim : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) u[i][e] = r1 * (u[i][e] - n[i][e] * dot1);
        Vec<IO, VEC>::store((IO *)a.dx + row * a.dim + c * VEC, u[i]);
      }
    }
  }
  write_partial<VEC, NV, BLOCK>(dw2, tm, a.dim, a.part[0], cols);
  if (a.w_post) write_partial<VEC, NV, BLOCK>(dw1, tm, a.dim, a.part[1], cols);
  if (a.scale) write_partial<VEC, NV, BLOCK>(ds, tm, a.dim, a.part[2], cols);
}

// out[c] = sum over the workgroups' partial rows, in a fixed order: 64 groups of
// rows side by side for 16 columns, then the groups' sums.  blockIdx.y picks the
// weight.  512 rows of 128 columns: 9.6 us with 16 groups for 64 columns, PARTIALS_US
// so.
__global__ __launch_bounds__(1024) void norm_partials_kernel(const float *part, int blocks, int dim, float *o0, float *o1,
                                                            float *o2) {
  __shared__ float lds[16][16];
  float *out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  const int c = blockIdx.x * 16 + (threadIdx.x & 15);
  float s = 0.0f;
  if (c < dim) {
    const float *p = part + (int64_t)blockIdx.y * blocks * dim + c;
#pragma unroll 8
    for (int b = threadIdx.x >> 4; b < blocks; b += 64) s += p[(int64_t)b * dim];
  }
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  if ((threadIdx.x & 63) < 16) lds[threadIdx.x >> 6][threadIdx.x & 15] = s;
  __syncthreads();
  if (threadIdx.x < 16 && c < dim) {
    s = 0.0f;
    for (int i = 0; i < 16; ++i) s += lds[i][threadIdx.x];
    out[c] = s;
  }
}

// the smallest power of two of at least n
int pow2_at_least(int n) {
  int p = 1;
  while (p < n) p <<= 1;
  return p;
}

bool aligned(const void *p, int64_t stride, int elem) {
  return ((uintptr_t)p & 15) == 0 && (stride * elem) % 16 == 0;
}

// The shape of a team for rows of nv vectors.
struct TeamPlan {
  int team, nv, block;
};
// Forward: a wave holds a row of up to 256 vectors (4 a lane), for the fewest
// exchanges; longer rows take a workgroup.
TeamPlan plan_forward(int nv) {
  if (nv <= 256) {
    const int team = nv >= 64 ? 64 : pow2_at_least(nv);
    return {team, (nv + team - 1) / team, 0};
  }
  const int most = nv > 4096 ? 16 : 4;
  const int team = pow2_at_least((nv + most - 1) / most);
  return {team, (nv + team - 1) / team, 1};
}
// Reverse: the weights' sums stay in registers beside five inputs, so that a
// thread holds one vector where 1024 threads can hold the row.
TeamPlan plan_reverse(int nv) {
  int team = pow2_at_least(nv);
  if (team > 1024) team = 1024;
  return {team, (nv + team - 1) / team, team > 64};
}

}  // namespace

#define NORM_LAUNCH(NV, BLK, THREADS, KERNEL, ...)                                                 \
  KERNEL<__VA_ARGS__, NV, BLK, THREADS><<<grid, BLK ? p.team : 256, 0, st>>>(a, p.team)
// The last type argument is the vector's width: rows of more than 4 vectors a
// thread are those of single elements.
#define NORM_PICK_FORWARD(KERNEL, VEC, ...)                                                        \
  do {                                                                                             \
    if (!p.block && p.nv == 1) NORM_LAUNCH(1, false, 256, KERNEL, __VA_ARGS__, VEC);               \
    else if (!p.block && p.nv == 2) NORM_LAUNCH(2, false, 256, KERNEL, __VA_ARGS__, VEC);          \
    else if (!p.block) NORM_LAUNCH(4, false, 256, KERNEL, __VA_ARGS__, VEC);                       \
    else if (p.nv <= 4) NORM_LAUNCH(4, true, 1024, KERNEL, __VA_ARGS__, VEC);                      \
    else if constexpr (VEC == 1) NORM_LAUNCH(16, true, 1024, KERNEL, __VA_ARGS__, VEC);            \
  } while (0)
// A thread of the reverse modes holds 8 elements of a row without spilling; 16 (rows
// of more than 8192) spill.
#define NORM_PICK_REVERSE(KERNEL, VEC, ...)                                                        \
  do {                                                                                             \
    if (grid == 0) break; /* no rows: the weights' sums are still written */                       \
    if (!p.block) NORM_LAUNCH(1, false, 256, KERNEL, __VA_ARGS__, VEC);                            \
    else if (p.team <= 256) NORM_LAUNCH(1, true, 256, KERNEL, __VA_ARGS__, VEC);                   \
    else if (p.nv == 1) NORM_LAUNCH(1, true, 1024, KERNEL, __VA_ARGS__, VEC);                      \
    else if (p.nv == 2) NORM_LAUNCH(2, true, 1024, KERNEL, __VA_ARGS__, VEC);                      \
    else if constexpr (VEC < 8) {                                                                  \
      if (p.nv <= 4) NORM_LAUNCH(4, true, 1024, KERNEL, __VA_ARGS__, VEC);                         \
      else if constexpr (VEC == 1) {                                                               \
        if (p.nv <= 8) NORM_LAUNCH(8, true, 1024, KERNEL, __VA_ARGS__, VEC);                       \
        else NORM_LAUNCH(16, true, 1024, KERNEL, __VA_ARGS__, VEC);                                \
      }                                                                                            \
    }                                                                                              \
  } while (0)

static int row_blocks(int64_t rows, const TeamPlan &p, int64_t most) {
  const int64_t per = p.block ? 1 : 256 / p.team;
  const int64_t n = (rows + per - 1) / per;
  return (int)(n < most ? n : most);
}

// Workgroups of a reverse mode: one alone where it passes the rows in four steps
// (its sums are the weights' gradients: no second launch), else up to `most`.
static int reverse_blocks(int64_t rows, const TeamPlan &p, int64_t most) {
  const int64_t per = p.block ? 1 : 256 / p.team;
  if (rows > 0 && rows <= 4 * per) return 1;
  if (p.team >= 512) most = most < 256 * (1024 / p.team) ? most : 256 * (1024 / p.team);
  return row_blocks(rows, p, most);
}

hipError_t launch_gated_norm(const GatedNormArgs &a, hipStream_t st) {
  const int64_t rows = a.tokens * a.heads;
  const int e = a.bf16 ? 2 : 4, vec = 16 / e;
  const bool wide = a.dim % vec == 0 && aligned(a.x, a.x_stride, e) && aligned(a.y, a.dim, e) &&
                    aligned(a.weight, 4, 4) && (a.act < 0 || aligned(a.gate, a.gate_stride, e));
  const TeamPlan p = plan_forward(wide ? a.dim / vec : a.dim);
  const int grid = row_blocks(rows, p, 1 << 20);
  TimedLaunch tl(K_NORM, st);
  if (a.bf16) {
    if (wide) NORM_PICK_FORWARD(gated_norm_kernel, 8, u16);
    else NORM_PICK_FORWARD(gated_norm_kernel, 1, u16);
  } else {
    if (wide) NORM_PICK_FORWARD(gated_norm_kernel, 4, float);
    else NORM_PICK_FORWARD(gated_norm_kernel, 1, float);
  }
  return hipGetLastError();
}

hipError_t launch_gated_norm_bwd(const GatedNormArgs &args, hipStream_t st) {
  GatedNormArgs a = args;
  const int64_t rows = a.tokens * a.heads;
  const int e = a.bf16 ? 2 : 4, vec = 16 / e;
  const bool wide = a.dim % vec == 0 && aligned(a.x, a.x_stride, e) && aligned(a.dy, a.dy_stride, e) &&
                    aligned(a.dx, a.dim, e) && aligned(a.weight, 4, 4) && aligned(a.dweight, a.dim, 4) &&
                    (a.act < 0 || (aligned(a.gate, a.gate_stride, e) && aligned(a.dgate, a.dim, e)));
  const TeamPlan p = plan_reverse(wide ? a.dim / vec : a.dim);
  const int grid = reverse_blocks(rows, p, norm_bwd_blocks(rows, a.dim));
  float *const part = a.part;
  if (grid == 1) a.part = a.dweight;
  TimedLaunch tl(K_NORM_BWD, st);
  if (a.bf16) {
    if (wide) NORM_PICK_REVERSE(gated_norm_bwd_kernel, 8, u16);
    else NORM_PICK_REVERSE(gated_norm_bwd_kernel, 1, u16);
  } else {
    if (wide) NORM_PICK_REVERSE(gated_norm_bwd_kernel, 4, float);
    else NORM_PICK_REVERSE(gated_norm_bwd_kernel, 1, float);
  }
  if (grid != 1)
    norm_partials_kernel<<<dim3((a.dim + 15) / 16, 1), 1024, 0, st>>>(part, grid, a.dim, a.dweight, nullptr, nullptr);
  return hipGetLastError();
}

hipError_t launch_residual_norm(const ResidualNormArgs &a, hipStream_t st) {
  const int e = a.bf16 ? 2 : 4, re = a.res_bf16 ? 2 : 4, vec = 16 / e;
  const bool wide = a.dim % vec == 0 && aligned(a.x, a.x_stride, e) && aligned(a.residual, a.dim, re) &&
                    aligned(a.h, a.dim, re) && aligned(a.y, a.dim, e) && aligned(a.w_pre, 4, 4) &&
                    (!a.w_post || aligned(a.w_post, 4, 4)) && (!a.scale || aligned(a.scale, 4, 4)) &&
                    (a.act < 0 || aligned(a.gate, a.gate_stride, e));
  const TeamPlan p = plan_forward(wide ? a.dim / vec : a.dim);
  const int grid = row_blocks(a.tokens, p, 1 << 20);
  TimedLaunch tl(K_NORM, st);
  if (a.bf16) {
    if (a.res_bf16) {
      if (wide) NORM_PICK_FORWARD(residual_norm_kernel, 8, u16, u16);
      else NORM_PICK_FORWARD(residual_norm_kernel, 1, u16, u16);
    } else {
      if (wide) NORM_PICK_FORWARD(residual_norm_kernel, 8, u16, float);
      else NORM_PICK_FORWARD(residual_norm_kernel, 1, u16, float);
    }
  } else {
    if (wide) NORM_PICK_FORWARD(residual_norm_kernel, 4, float, float);
    else NORM_PICK_FORWARD(residual_norm_kernel, 1, float, float);
  }
  return hipGetLastError();
}

hipError_t launch_residual_norm_bwd(const ResidualNormArgs &args, hipStream_t st) {
  ResidualNormArgs a = args;
  const int e = a.bf16 ? 2 : 4, re = a.res_bf16 ? 2 : 4, vec = 16 / e;
  const bool wide = a.dim % vec == 0 && aligned(a.x, a.x_stride, e) && aligned(a.residual, a.dim, re) &&
                    aligned(a.dy, a.dim, e) && aligned(a.dx, a.dim, e) && aligned(a.dres, a.dim, re) &&
                    (!a.dh || aligned(a.dh, a.dim, re)) && aligned(a.dw_pre, a.dim, 4) &&
                    (!a.w_post || aligned(a.dw_post, a.dim, 4)) && (!a.scale || aligned(a.dscale, a.dim, 4)) && aligned(a.w_pre, 4, 4) &&
                    (!a.w_post || aligned(a.w_post, 4, 4)) && (!a.scale || aligned(a.scale, 4, 4)) &&
                    (a.act < 0 || (aligned(a.gate, a.gate_stride, e) && aligned(a.dgate, a.dim, e)));
  const TeamPlan p = plan_reverse(wide ? a.dim / vec : a.dim);
  const int grid = reverse_blocks(a.tokens, p, norm_bwd_blocks(a.tokens, a.dim));
  float *const part = a.part[0];
  a.part[1] = part + (int64_t)grid * a.dim;
  a.part[2] = part + 2 * (int64_t)grid * a.dim;
  if (grid == 1) {
    a.part[0] = a.dw_pre;
    a.part[1] = a.dw_post;
    a.part[2] = a.dscale;
  }
  TimedLaunch tl(K_NORM_BWD, st);
  if (a.bf16) {
    if (a.res_bf16) {
      if (wide) NORM_PICK_REVERSE(residual_norm_bwd_kernel, 8, u16, u16);
      else NORM_PICK_REVERSE(residual_norm_bwd_kernel, 1, u16, u16);
    } else {
      if (wide) NORM_PICK_REVERSE(residual_norm_bwd_kernel, 8, u16, float);
      else NORM_PICK_REVERSE(residual_norm_bwd_kernel, 1, u16, float);
    }
  } else {
    if (wide) NORM_PICK_REVERSE(residual_norm_bwd_kernel, 4, float, float);
    else NORM_PICK_REVERSE(residual_norm_bwd_kernel, 1, float, float);
  }
  if (grid != 1)
    norm_partials_kernel<<<dim3((a.dim + 15) / 16, 3), 1024, 0, st>>>(
        part, grid, a.dim, a.dw_pre, a.w_post ? a.dw_post : nullptr, a.scale ? a.dscale : nullptr);
  return hipGetLastError();
}

}  // namespace flare
