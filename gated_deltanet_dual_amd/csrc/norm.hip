// norm.hip -- the norms before and after a block, fused with its gate and
// residual scale, forward and reverse mode.
//
//   gated norm     y = x r w act(g),  r = 1 / sqrt(mean x^2 + eps), per head row
//   residual norm  n = x r1 w1 (or x);  h = res + s act(g) n;  y = h r2 w2
//
// Reverse of a normalised row u = x r with incoming gradient du:
//   dx = r (du - u mean(du u)).
//
// Memory bounds all of them: a row is read once, held in registers in fp32 through
// its reductions, and written once; each rounding to bf16 is that of an output.
// Small launches (up to a few hundred rows) take the 4 us of a launch.
#include <hip/hip_runtime.h>

#include "layer_launch.h"
#include "vec_io.h"

namespace flare {
namespace {

// exp(-g) = 2^hi 2^lo with hi the rounded product -g log2 e and lo what its rounding and
// the constant's left over: off by 4 half steps for every g, where 2^hi alone is off by |g|
// of them.  A product beyond every exponent (or NaN) has no rest to add.  (32768 x 16 rows
// of 128, both directions: 210 us with the rest and without, 214 with the library's expf.)
__device__ __forceinline__ float exp_minus(float g) {
  constexpr float kLog2e = 1.44269504088896340736, kLog2eRest = 1.44269504088896340736 - (double)kLog2e;
  const float hi = -g * kLog2e, rest = __builtin_fmaf(-g, kLog2eRest, __builtin_fmaf(-g, kLog2e, -hi));
  return __builtin_amdgcn_exp2f(hi) * __builtin_fmaf(fabsf(hi) < 256.0f ? rest : 0.0f, 0.69314718055994530942f, 1.0f);
}
__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + exp_minus(g)); }

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
// The vector c of an fp32 weight, n of it, or ones where it is absent.
template <int VEC, bool TAIL> __device__ __forceinline__ void load_or_one(const float *w, int c, int n, float *f) {
  if (w) {
    load_vec<float, VEC, TAIL>(w + c * VEC, n, f);
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
// 32768 x 16 rows of 128, bf16: 403 MB in 79 to 82 us, 4.9 to 5.1 TB/s (a copy of that
// size reaches 5.1 to 5.5).
template <typename IO, int VEC, bool TAIL, int NV, bool BLOCK, int THREADS>
__global__ __launch_bounds__(THREADS) void gated_norm_kernel(GatedNormArgs a, int team) {
  __shared__ float red[16];
  const Team<BLOCK> tm{team, BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (team - 1))};
  const int per = BLOCK ? 1 : blockDim.x / team;
  const uint32_t rows = (uint32_t)(a.tokens * a.heads);
  const int nv = (a.dim + VEC - 1) / VEC;
  for (uint32_t row = blockIdx.x * per + (BLOCK ? 0 : threadIdx.x / team); row < rows; row += gridDim.x * per) {
    const uint32_t t = row / (uint32_t)a.heads, h = row - t * (uint32_t)a.heads;
    const IO *x = (const IO *)a.x + (int64_t)t * a.x_stride + (int64_t)h * a.dim;
    const IO *g = (const IO *)a.gate + (int64_t)t * a.gate_stride + (int64_t)h * a.dim;
    float xv[NV][VEC], gv[NV][VEC], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        load_vec<IO, VEC, TAIL>(x + c * VEC, a.dim - c * VEC, xv[i]);
        if (a.act >= 0) load_vec<IO, VEC, TAIL>(g + c * VEC, a.dim - c * VEC, gv[i]);
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
        load_vec<float, VEC, TAIL>(a.weight + c * VEC, a.dim - c * VEC, w);
        gate_values<VEC>(gv[i], a.act, o);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] *= xv[i][e] * r * w[e];
        store_vec<IO, VEC, TAIL>(y + c * VEC, a.dim - c * VEC, o);
      }
    }
  }
}

// Adds the threads' column sums of a workgroup: `acc` of every team for the
// vectors it holds, into part[blockIdx.x][dim].
template <int VEC, bool TAIL, int NV, bool BLOCK>
__device__ __forceinline__ void write_partial(const float (&acc)[NV][VEC], const Team<BLOCK> &tm, int dim, float *part,
                                              float *lds) {
  const int nv = (dim + VEC - 1) / VEC;
  float *out = part + (int64_t)blockIdx.x * dim;
  if constexpr (BLOCK) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * tm.size;
      if (c < nv) store_vec<float, VEC, TAIL>(out + c * VEC, dim - c * VEC, acc[i]);
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
        if (c < dim) {
          float s = 0.0f;
          for (int k = 0; k < teams; ++k) s += lds[k * tm.size * VEC + j];
          out[c] = s;
        }
      }
    }
  }
}

// A workgroup keeps its rows' share of the weight's gradient in registers over all its
// rows and writes it once; a second launch adds the workgroups' up in a fixed order.
// 32768 x 16 rows of 128, bf16: 671 MB in 125 us, 5.4 TB/s.
template <typename IO, int VEC, bool TAIL, int NV, bool BLOCK, int THREADS>
__global__ __launch_bounds__(THREADS) void gated_norm_bwd_kernel(GatedNormArgs a, int team) {
  __shared__ float red[16];
  __shared__ float cols[BLOCK ? 1 : 256 * VEC];
  const Team<BLOCK> tm{team, BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (team - 1))};
  const int per = BLOCK ? 1 : blockDim.x / team;
  const uint32_t rows = (uint32_t)(a.tokens * a.heads);
  const int nv = (a.dim + VEC - 1) / VEC;
  float dw[NV][VEC] = {};
  float w[NV][VEC] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (const int c = tm.lane + i * team; c < nv) load_vec<float, VEC, TAIL>(a.weight + c * VEC, a.dim - c * VEC, w[i]);
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
        load_vec<IO, VEC, TAIL>(x + c * VEC, a.dim - c * VEC, u[i]);
        load_vec<IO, VEC, TAIL>(dy + c * VEC, a.dim - c * VEC, du[i]);
        if (a.act >= 0) load_vec<IO, VEC, TAIL>(g + c * VEC, a.dim - c * VEC, gv[i]);
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
        store_vec<IO, VEC, TAIL>((IO *)a.dx + (int64_t)row * a.dim + c * VEC, a.dim - c * VEC, o);
        if (a.act >= 0) store_vec<IO, VEC, TAIL>((IO *)a.dgate + (int64_t)row * a.dim + c * VEC, a.dim - c * VEC, gv[i]);
      }
    }
  }
  write_partial<VEC, TAIL, NV, BLOCK>(dw, tm, a.dim, a.part, cols);
}

// ---------------------------------------------------------------- residual norm
// 32768 rows of 2048, bf16 with an fp32 residual, gate, post-norm and scale: 940 MB in
// 182 us, 5.2 TB/s.
template <typename IO, typename RES, int VEC, bool TAIL, int NV, bool BLOCK, int THREADS>
__global__ __launch_bounds__(THREADS) void residual_norm_kernel(ResidualNormArgs a, int team) {
  __shared__ float red[16];
  const Team<BLOCK> tm{team, BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (team - 1))};
  const int per = BLOCK ? 1 : blockDim.x / team;
  const int nv = (a.dim + VEC - 1) / VEC;
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
        load_vec<IO, VEC, TAIL>(x + c * VEC, a.dim - c * VEC, xv[i]);
        load_vec<RES, VEC, TAIL>(res + c * VEC, a.dim - c * VEC, hv[i]);
        if (a.act >= 0) load_vec<IO, VEC, TAIL>(g + c * VEC, a.dim - c * VEC, gv[i]);
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
        load_or_one<VEC, TAIL>(a.w_post, c, a.dim - c * VEC, w1);
        load_or_one<VEC, TAIL>(a.scale, c, a.dim - c * VEC, sc);
        gate_values<VEC>(gv[i], a.act, f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          hv[i][e] += xv[i][e] * r1 * w1[e] * f[e] * sc[e];
          ss += hv[i][e] * hv[i][e];
        }
        store_vec<RES, VEC, TAIL>((RES *)a.h + row * a.dim + c * VEC, a.dim - c * VEC, hv[i]);
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
        load_vec<float, VEC, TAIL>(a.w_pre + c * VEC, a.dim - c * VEC, w2);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = hv[i][e] * r2 * w2[e];
        store_vec<IO, VEC, TAIL>((IO *)a.y + row * a.dim + c * VEC, a.dim - c * VEC, o);
      }
    }
  }
}

// h is formed again from the inputs: storing the fp32 h would be read instead of x,
// the gate and the residual, which their own gradients need anyway.  All weights' sums
// in registers, as above.  32768 rows of 2048, bf16 with an fp32 residual and all
// options: 1.48 GB in 275 us, 5.4 TB/s.
template <typename IO, typename RES, int VEC, bool TAIL, int NV, bool BLOCK, int THREADS>
__global__ __launch_bounds__(THREADS) void residual_norm_bwd_kernel(ResidualNormArgs a, int team) {
  __shared__ float red[16];
  __shared__ float cols[BLOCK ? 1 : 256 * VEC];
  const Team<BLOCK> tm{team, BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (team - 1))};
  const int per = BLOCK ? 1 : blockDim.x / team;
  const int nv = (a.dim + VEC - 1) / VEC;
  float dw2[NV][VEC] = {}, dw1[NV][VEC] = {}, ds[NV][VEC] = {};
  // the weights of a thread's one vector stay in registers over its rows (of 128
  // registers that larger workgroups leave, they would be 3 VEC too many)
  constexpr bool KEEP = NV == 1 && THREADS <= 256;
  float w2[VEC] = {}, w1[VEC] = {}, sc[VEC] = {};
  if (KEEP && tm.lane < nv) {
    const int c = tm.lane;
    load_vec<float, VEC, TAIL>(a.w_pre + c * VEC, a.dim - c * VEC, w2);
    load_or_one<VEC, TAIL>(a.w_post, c, a.dim - c * VEC, w1);
    load_or_one<VEC, TAIL>(a.scale, c, a.dim - c * VEC, sc);
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
        load_vec<IO, VEC, TAIL>(x + c * VEC, a.dim - c * VEC, n[i]);
        load_vec<RES, VEC, TAIL>(res + c * VEC, a.dim - c * VEC, u[i]);
        load_vec<IO, VEC, TAIL>((const IO *)a.dy + row * a.dim + c * VEC, a.dim - c * VEC, dy[i]);
        if (a.act >= 0) load_vec<IO, VEC, TAIL>(g + c * VEC, a.dim - c * VEC, f[i]);
        if (a.dh) {
          load_vec<RES, VEC, TAIL>((const RES *)a.dh + row * a.dim + c * VEC, a.dim - c * VEC, dh[i]);
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
          load_vec<float, VEC, TAIL>(a.w_pre + c * VEC, a.dim - c * VEC, w2);
          load_or_one<VEC, TAIL>(a.w_post, c, a.dim - c * VEC, w1);
          load_or_one<VEC, TAIL>(a.scale, c, a.dim - c * VEC, sc);
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
          load_or_one<VEC, TAIL>(a.w_post, c, a.dim - c * VEC, w1);
          load_or_one<VEC, TAIL>(a.scale, c, a.dim - c * VEC, sc);
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
        store_vec<RES, VEC, TAIL>((RES *)a.dres + row * a.dim + c * VEC, a.dim - c * VEC, dh[i]);
        if (a.act >= 0) store_vec<IO, VEC, TAIL>((IO *)a.dgate + row * a.dim + c * VEC, a.dim - c * VEC, df[i]);
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
        store_vec<IO, VEC, TAIL>((IO *)a.dx + row * a.dim + c * VEC, a.dim - c * VEC, u[i]);
      }
    }
  }
  write_partial<VEC, TAIL, NV, BLOCK>(dw2, tm, a.dim, a.part[0], cols);
  if (a.w_post) write_partial<VEC, TAIL, NV, BLOCK>(dw1, tm, a.dim, a.part[1], cols);
  if (a.scale) write_partial<VEC, TAIL, NV, BLOCK>(ds, tm, a.dim, a.part[2], cols);
}

// out[c] = sum over the workgroups' partial rows, in a fixed order: 64 groups of
// rows side by side for 16 columns, then the groups' sums.  blockIdx.y picks the
// weight.  A launch and its reads' latency: 1536 rows of 128 columns 9.6 us with 16
// groups for 64 columns, 4.6 us so.
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

// The shape of a team for rows of nv vectors of `vec` elements.
struct TeamPlan {
  int team, nv;
  int threads;  // 0: teams of up to a wave, in workgroups of 256; else the row's workgroup is of at most so many
};
// Forward: a wave holds a row of up to 256 vectors (4 a lane), for the fewest
// exchanges; then 256 threads, 4 vectors each (4096 x 4096 bf16: 30 us, where 1024
// threads of one vector take 85).
TeamPlan plan_forward(int nv) {
  if (nv <= 256) {
    const int team = nv >= 64 ? 64 : pow2_at_least(nv);
    return {team, (nv + team - 1) / team, 0};
  }
  const int team = nv <= 1024 ? 256 : 1024;
  return {team, (nv + team - 1) / team, team};
}
// Reverse: the weights' sums stay in registers beside five inputs, so that a
// thread holds 8 elements, or 16 where it has 256 registers (512 threads); rows
// of more than 8192 spill.
TeamPlan plan_reverse(int nv, int vec) {
  const int one = 8 / vec;  // vectors of 8 elements
  if (nv <= 64 * one) {
    const int team = nv >= 64 ? 64 : pow2_at_least(nv);
    return {team, (nv + team - 1) / team, 0};
  }
  int team;
  if (nv <= 256 * one) team = pow2_at_least((nv + one - 1) / one);
  else if (nv <= 512 * one) team = vec == 8 ? 256 : 512;
  else team = vec == 8 && nv <= 1024 ? 512 : 1024;
  return {team, (nv + team - 1) / team, team <= 256 ? 256 : team};
}

int row_blocks(int64_t rows, const TeamPlan &p, int64_t most) {
  const int64_t per = p.threads ? 1 : 256 / p.team;
  const int64_t n = (rows + per - 1) / per;
  return (int)(n < most ? n : most);
}

// Workgroups of a reverse mode: one alone where it passes the rows in four steps
// (its sums are the weights' gradients: no second launch), else up to `most` or
// what the chip holds at a time.
int reverse_blocks(int64_t rows, const TeamPlan &p, int64_t most) {
  const int64_t per = p.threads ? 1 : 256 / p.team;
  if (rows > 0 && rows <= 4 * per) return 1;
  const int64_t hold = p.threads == 0 ? 1536 : p.threads > 256 ? 256 : p.nv > 1 ? 512 : 768 * (256 / p.team);
  return row_blocks(rows, p, most < hold ? most : hold);
}

template <int VEC, bool TAIL> struct Width {
  static constexpr int vec = VEC;
  static constexpr bool tail = TAIL;
};
// f(Width<VEC, TAIL>) for rows of `dim` channels
template <int VEC, typename F> void with_width(int dim, F f) {
  if (dim % VEC == 0) f(Width<VEC, false>{});
  else f(Width<VEC, true>{});
}

// LAUNCH(vectors a thread, a workgroup holds the row, its threads at most)
#define NORM_FORWARD(LAUNCH)                                                    \
  do {                                                                          \
    if (p.threads == 0 && p.nv == 1) LAUNCH(1, false, 256);                     \
    else if (p.threads == 0 && p.nv == 2) LAUNCH(2, false, 256);                \
    else if (p.threads == 0) LAUNCH(4, false, 256);                             \
    else if (p.threads == 256) LAUNCH(4, true, 256);                            \
    else if (p.nv == 2) LAUNCH(2, true, 1024);                                  \
    else if constexpr (W::vec < 8) LAUNCH(4, true, 1024);                       \
  } while (0)
#define NORM_REVERSE(LAUNCH)                                                    \
  do {                                                                          \
    if (grid == 0) break; /* no rows: the weights' sums are still written */    \
    if (p.threads == 0 && p.nv == 1) LAUNCH(1, false, 256);                     \
    else if (p.threads == 256 && p.nv == 2) LAUNCH(2, true, 256);               \
    else if (p.threads == 512) LAUNCH(2, true, 512);                            \
    else if (p.threads == 1024 && p.nv == 2) LAUNCH(2, true, 1024);             \
    else if constexpr (W::vec < 8) {                                            \
      if (p.threads == 0) LAUNCH(2, false, 256);                                \
      else LAUNCH(4, true, 1024);                                               \
    } else LAUNCH(1, true, 256); /* fp32's are of two vectors a thread */       \
  } while (0)

template <typename IO, int VEC> void gated_forward(const GatedNormArgs &a, hipStream_t st) {
  const TeamPlan p = plan_forward((a.dim + VEC - 1) / VEC);
  const int grid = row_blocks(a.tokens * a.heads, p, 1 << 20);
  with_width<VEC>(a.dim, [&](auto w) {
    using W = decltype(w);
#define LAUNCH(NV, BLK, N) \
  gated_norm_kernel<IO, W::vec, W::tail, NV, BLK, N><<<grid, BLK ? p.team : 256, 0, st>>>(a, p.team)
    NORM_FORWARD(LAUNCH);
#undef LAUNCH
  });
}

template <typename IO, int VEC> hipError_t gated_reverse(GatedNormArgs a, hipStream_t st) {
  const int64_t rows = a.tokens * a.heads;
  const TeamPlan p = plan_reverse((a.dim + VEC - 1) / VEC, VEC);
  const int grid = reverse_blocks(rows, p, norm_bwd_blocks(rows, a.dim));
  float *const part = a.part;
  if (grid == 1) a.part = a.dweight;
  with_width<VEC>(a.dim, [&](auto w) {
    using W = decltype(w);
#define LAUNCH(NV, BLK, N) \
  gated_norm_bwd_kernel<IO, W::vec, W::tail, NV, BLK, N><<<grid, BLK ? p.team : 256, 0, st>>>(a, p.team)
    NORM_REVERSE(LAUNCH);
#undef LAUNCH
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (grid != 1)
    norm_partials_kernel<<<dim3((a.dim + 15) / 16, 1), 1024, 0, st>>>(part, grid, a.dim, a.dweight, nullptr, nullptr);
  return hipGetLastError();
}

template <typename IO, typename RES, int VEC> void residual_forward(const ResidualNormArgs &a, hipStream_t st) {
  const TeamPlan p = plan_forward((a.dim + VEC - 1) / VEC);
  const int grid = row_blocks(a.tokens, p, 1 << 20);
  with_width<VEC>(a.dim, [&](auto w) {
    using W = decltype(w);
#define LAUNCH(NV, BLK, N) \
  residual_norm_kernel<IO, RES, W::vec, W::tail, NV, BLK, N><<<grid, BLK ? p.team : 256, 0, st>>>(a, p.team)
    NORM_FORWARD(LAUNCH);
#undef LAUNCH
  });
}

template <typename IO, typename RES, int VEC> hipError_t residual_reverse(ResidualNormArgs a, hipStream_t st) {
  const TeamPlan p = plan_reverse((a.dim + VEC - 1) / VEC, VEC);
  const int grid = reverse_blocks(a.tokens, p, norm_bwd_blocks(a.tokens, a.dim));
  float *const part = a.part[0];
  a.part[1] = part + (int64_t)grid * a.dim;
  a.part[2] = part + 2 * (int64_t)grid * a.dim;
  if (grid == 1) {
    a.part[0] = a.dw_pre;
    a.part[1] = a.dw_post;
    a.part[2] = a.dscale;
  }
  with_width<VEC>(a.dim, [&](auto w) {
    using W = decltype(w);
#define LAUNCH(NV, BLK, N) \
  residual_norm_bwd_kernel<IO, RES, W::vec, W::tail, NV, BLK, N><<<grid, BLK ? p.team : 256, 0, st>>>(a, p.team)
    NORM_REVERSE(LAUNCH);
#undef LAUNCH
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (grid != 1)
    norm_partials_kernel<<<dim3((a.dim + 15) / 16, 3), 1024, 0, st>>>(
        part, grid, a.dim, a.dw_pre, a.w_post ? a.dw_post : nullptr, a.scale ? a.dscale : nullptr);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_norm(const GatedNormArgs &a, hipStream_t st) {
  TimedLaunch tl(K_NORM, st);
  if (a.bf16) gated_forward<u16, 8>(a, st);
  else gated_forward<float, 4>(a, st);
  return hipGetLastError();
}

hipError_t launch_gated_norm_bwd(const GatedNormArgs &a, hipStream_t st) {
  TimedLaunch tl(K_NORM_BWD, st);
  return a.bf16 ? gated_reverse<u16, 8>(a, st) : gated_reverse<float, 4>(a, st);
}

hipError_t launch_residual_norm(const ResidualNormArgs &a, hipStream_t st) {
  TimedLaunch tl(K_NORM, st);
  if (a.bf16 && a.res_bf16) residual_forward<u16, u16, 8>(a, st);
  else if (a.bf16) residual_forward<u16, float, 8>(a, st);
  else residual_forward<float, float, 4>(a, st);
  return hipGetLastError();
}

hipError_t launch_residual_norm_bwd(const ResidualNormArgs &a, hipStream_t st) {
  TimedLaunch tl(K_NORM_BWD, st);
  if (a.bf16 && a.res_bf16) return residual_reverse<u16, u16, 8>(a, st);
  return a.bf16 ? residual_reverse<u16, float, 8>(a, st) : residual_reverse<float, float, 4>(a, st);
}

}  // namespace flare
