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

// act(g); act < 0: no gate
__device__ __forceinline__ float gate_value(float g, int act) {
  if (act == FLARE_GATE_LINEAR) return g;
  const float p = sigmoid(g);
  return act == FLARE_GATE_SIGMOID ? p : g * p;
}
// act(g) and its derivative
__device__ __forceinline__ float gate_value_d(float g, int act, float &d) {
  if (act == FLARE_GATE_LINEAR) {
    d = 1.0f;
    return g;
  }
  const float p = sigmoid(g);
  if (act == FLARE_GATE_SIGMOID) {
    d = p * (1.0f - p);
    return p;
  }
  d = p * (1.0f + g * (1.0f - p));
  return g * p;
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
template <typename IO, int VEC, int NV, bool BLOCK>
__global__ __launch_bounds__(BLOCK ? 1024 : 256) void gated_norm_kernel(GatedNormArgs a, int team) {
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
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          o[e] = xv[i][e] * r * w[e];
          if (a.act >= 0) o[e] *= gate_value(gv[i][e], a.act);
        }
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

template <typename IO, int VEC, int NV, bool BLOCK>
__global__ __launch_bounds__(BLOCK ? 1024 : 256) void gated_norm_bwd_kernel(GatedNormArgs a, int team) {
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
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          u[i][e] *= r;
          float d = 0.0f, act = 1.0f;
          if (a.act >= 0) act = gate_value_d(gv[i][e], a.act, d);
          const float dn = du[i][e];
          dw[i][e] += dn * u[i][e] * act;
          gv[i][e] = dn * u[i][e] * w[i][e] * d;
          du[i][e] = dn * w[i][e] * act;
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
template <typename IO, typename RES, int VEC, int NV, bool BLOCK>
__global__ __launch_bounds__(BLOCK ? 1024 : 256) void residual_norm_kernel(ResidualNormArgs a, int team) {
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
        float w1[VEC], sc[VEC];
        if (a.w_post) Vec<float, VEC>::load(a.w_post + c * VEC, w1);
        if (a.scale) Vec<float, VEC>::load(a.scale + c * VEC, sc);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float z = xv[i][e];
          if (a.w_post) z *= r1 * w1[e];
          if (a.act >= 0) z *= gate_value(gv[i][e], a.act);
          if (a.scale) z *= sc[e];
          hv[i][e] += z;
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

template <typename IO, typename RES, int VEC, int NV, bool BLOCK>
__global__ __launch_bounds__(BLOCK ? 1024 : 256) void residual_norm_bwd_kernel(ResidualNormArgs a, int team) {
  __shared__ float red[16];
  __shared__ float cols[BLOCK ? 1 : 256 * VEC];
  const Team<BLOCK> tm{team, BLOCK ? (int)threadIdx.x : (int)(threadIdx.x & (team - 1))};
  const int per = BLOCK ? 1 : blockDim.x / team;
  const int nv = a.dim / VEC;
  float dw2[NV][VEC] = {}, dw1[NV][VEC] = {}, ds[NV][VEC] = {};
  for (int64_t row = (int64_t)blockIdx.x * per + (BLOCK ? 0 : threadIdx.x / team); row < a.tokens;
       row += (int64_t)gridDim.x * per) {
    const IO *x = (const IO *)a.x + row * a.x_stride;
    const IO *g = (const IO *)a.gate + row * a.gate_stride;
    const RES *res = (const RES *)a.residual + row * a.dim;
    const float r1 = a.rstd[2 * row], r2 = a.rstd[2 * row + 1];
    // h again, in fp32 as the forward formed it
    float n[NV][VEC], gv[NV][VEC], u[NV][VEC], dy[NV][VEC], dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        Vec<IO, VEC>::load(x + c * VEC, n[i]);
        Vec<RES, VEC>::load(res + c * VEC, u[i]);
        Vec<IO, VEC>::load((const IO *)a.dy + row * a.dim + c * VEC, dy[i]);
        if (a.act >= 0) Vec<IO, VEC>::load(g + c * VEC, gv[i]);
        float w1[VEC], w2[VEC], sc[VEC];
        Vec<float, VEC>::load(a.w_pre + c * VEC, w2);
        if (a.w_post) Vec<float, VEC>::load(a.w_post + c * VEC, w1);
        if (a.scale) Vec<float, VEC>::load(a.scale + c * VEC, sc);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float z = n[i][e];
          if (a.w_post) z *= r1 * w1[e];
          if (a.act >= 0) z *= gate_value(gv[i][e], a.act);
          if (a.scale) z *= sc[e];
          u[i][e] = (u[i][e] + z) * r2;
          dw2[i][e] += dy[i][e] * u[i][e];
          dy[i][e] *= w2[e];
          dot += dy[i][e] * u[i][e];
          n[i][e] *= r1;  // the normalised x (x itself without a post-norm)
        }
      }
    }
    dot = tm.sum(dot, red) / (float)a.dim;
    float dot1 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        float dh[VEC], w1[VEC], sc[VEC], dg[VEC];
        if (a.dh) Vec<RES, VEC>::load((const RES *)a.dh + row * a.dim + c * VEC, dh);
        if (a.w_post) Vec<float, VEC>::load(a.w_post + c * VEC, w1);
        if (a.scale) Vec<float, VEC>::load(a.scale + c * VEC, sc);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float d = r2 * (dy[i][e] - u[i][e] * dot);
          if (a.dh) d += dh[e];
          dh[e] = d;
          float act = 1.0f, dact = 0.0f;
          if (a.act >= 0) act = gate_value_d(gv[i][e], a.act, dact);
          const float z = a.w_post ? n[i][e] * w1[e] : n[i][e];
          const float s = a.scale ? sc[e] : 1.0f;
          dg[e] = d * s * z * dact;
          if (a.scale) ds[i][e] += d * act * z;
          d *= s * act;  // the gradient of z
          if (a.w_post) {
            dw1[i][e] += d * n[i][e];
            d *= w1[e];
            dot1 += d * n[i][e];
          }
          u[i][e] = d;
        }
        Vec<RES, VEC>::store((RES *)a.dres + row * a.dim + c * VEC, dh);
        if (a.act >= 0) Vec<IO, VEC>::store((IO *)a.dgate + row * a.dim + c * VEC, dg);
      }
    }
    if (a.w_post) dot1 = tm.sum(dot1, red) / (float)a.dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tm.lane + i * team;
      if (c < nv) {
        if (a.w_post) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) u[i][e] = r1 * (u[i][e] - n[i][e] * dot1);
        }
        Vec<IO, VEC>::store((IO *)a.dx + row * a.dim + c * VEC, u[i]);
      }
    }
  }
  const int64_t plane = (int64_t)gridDim.x * a.dim;
  write_partial<VEC, NV, BLOCK>(dw2, tm, a.dim, a.part, cols);
  if (a.w_post) write_partial<VEC, NV, BLOCK>(dw1, tm, a.dim, a.part + plane, cols);
  if (a.scale) write_partial<VEC, NV, BLOCK>(ds, tm, a.dim, a.part + 2 * plane, cols);
}

// out[c] = sum over the blocks' partial rows, in a fixed order: 16 groups of
// rows side by side, then the groups' sums.  blockIdx.y picks the weight.
__global__ void norm_partials_kernel(const float *part, int blocks, int dim, float *o0, float *o1, float *o2) {
  __shared__ float lds[16][64];
  float *out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
  float s = 0.0f;
  if (c < dim) {
    const float *p = part + (int64_t)blockIdx.y * blocks * dim + c;
    for (int b = w; b < blocks; b += 16) s += p[(int64_t)b * dim];
  }
  lds[w][threadIdx.x & 63] = s;
  __syncthreads();
  if (w == 0 && c < dim) {
    s = 0.0f;
    for (int i = 0; i < 16; ++i) s += lds[i][threadIdx.x & 63];
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

// The shape of a team for rows of nv vectors: `max_nv` vectors a thread at
// most, a wave if that holds the row.
struct TeamPlan {
  int team, nv, block;
};
TeamPlan plan_team(int nv, int max_nv) {
  const int wave = pow2_at_least((nv + max_nv - 1) / max_nv);
  if (wave <= 64) {
    // as many lanes as there are vectors, up to a wave; then more vectors a lane
    const int team = nv >= 64 ? 64 : pow2_at_least(nv);
    return {team, (nv + team - 1) / team, 0};
  }
  return {wave, (nv + wave - 1) / wave, 1};
}

}  // namespace

#define NORM_LAUNCH(NV, BLK, KERNEL, ...)                                                          \
  KERNEL<__VA_ARGS__, NV, BLK><<<grid, BLK ? p.team : 256, 0, st>>>(a, p.team)
#define NORM_PICK(KERNEL, ...)                                                                     \
  do {                                                                                             \
    if (grid == 0) break; /* no rows: the reverse modes still write their weights' sums */         \
    if (p.block) {                                                                                 \
      if (p.nv <= 4) NORM_LAUNCH(4, true, KERNEL, __VA_ARGS__);                                    \
      else NORM_LAUNCH(16, true, KERNEL, __VA_ARGS__);                                             \
    } else if (p.nv == 1) NORM_LAUNCH(1, false, KERNEL, __VA_ARGS__);                              \
    else if (p.nv == 2) NORM_LAUNCH(2, false, KERNEL, __VA_ARGS__);                                \
    else NORM_LAUNCH(4, false, KERNEL, __VA_ARGS__);                                               \
  } while (0)

// vectors a thread holds at most: 4, or 16 single elements where the row
// needs more than 1024 threads of 4
static TeamPlan plan_rows(int nv) { return plan_team(nv, nv > 4096 ? 16 : 4); }

static int row_blocks(int64_t rows, const TeamPlan &p, int64_t most) {
  const int64_t per = p.block ? 1 : 256 / p.team;
  const int64_t n = (rows + per - 1) / per;
  return (int)(n < most ? n : most);
}

hipError_t launch_gated_norm(const GatedNormArgs &a, hipStream_t st) {
  const int64_t rows = a.tokens * a.heads;
  const int e = a.bf16 ? 2 : 4, vec = 16 / e;
  const bool wide = a.dim % vec == 0 && aligned(a.x, a.x_stride, e) && aligned(a.y, a.dim, e) &&
                    aligned(a.weight, 4, 4) && (a.act < 0 || aligned(a.gate, a.gate_stride, e));
  const TeamPlan p = plan_rows(wide ? a.dim / vec : a.dim);
  const int grid = row_blocks(rows, p, 1 << 20);
  TimedLaunch tl(K_NORM, st);
  if (a.bf16) {
    if (wide) NORM_PICK(gated_norm_kernel, u16, 8);
    else NORM_PICK(gated_norm_kernel, u16, 1);
  } else {
    if (wide) NORM_PICK(gated_norm_kernel, float, 4);
    else NORM_PICK(gated_norm_kernel, float, 1);
  }
  return hipGetLastError();
}

hipError_t launch_gated_norm_bwd(const GatedNormArgs &a, hipStream_t st) {
  const int64_t rows = a.tokens * a.heads;
  const int e = a.bf16 ? 2 : 4, vec = 16 / e;
  const bool wide = a.dim % vec == 0 && aligned(a.x, a.x_stride, e) && aligned(a.dy, a.dy_stride, e) &&
                    aligned(a.dx, a.dim, e) && aligned(a.weight, 4, 4) && aligned(a.part, a.dim, 4) &&
                    (a.act < 0 || (aligned(a.gate, a.gate_stride, e) && aligned(a.dgate, a.dim, e)));
  const TeamPlan p = plan_rows(wide ? a.dim / vec : a.dim);
  const int grid = row_blocks(rows, p, norm_bwd_blocks(rows));
  TimedLaunch tl(K_NORM_BWD, st);
  if (a.bf16) {
    if (wide) NORM_PICK(gated_norm_bwd_kernel, u16, 8);
    else NORM_PICK(gated_norm_bwd_kernel, u16, 1);
  } else {
    if (wide) NORM_PICK(gated_norm_bwd_kernel, float, 4);
    else NORM_PICK(gated_norm_bwd_kernel, float, 1);
  }
  norm_partials_kernel<<<dim3((a.dim + 63) / 64, 1), 1024, 0, st>>>(a.part, grid, a.dim, a.dweight, nullptr, nullptr);
  return hipGetLastError();
}

hipError_t launch_residual_norm(const ResidualNormArgs &a, hipStream_t st) {
  const int e = a.bf16 ? 2 : 4, re = a.res_bf16 ? 2 : 4, vec = 16 / e;
  const bool wide = a.dim % vec == 0 && aligned(a.x, a.x_stride, e) && aligned(a.residual, a.dim, re) &&
                    aligned(a.h, a.dim, re) && aligned(a.y, a.dim, e) && aligned(a.w_pre, 4, 4) &&
                    (!a.w_post || aligned(a.w_post, 4, 4)) && (!a.scale || aligned(a.scale, 4, 4)) &&
                    (a.act < 0 || aligned(a.gate, a.gate_stride, e));
  const TeamPlan p = plan_rows(wide ? a.dim / vec : a.dim);
  const int grid = row_blocks(a.tokens, p, 1 << 20);
  TimedLaunch tl(K_NORM, st);
  if (a.bf16) {
    if (a.res_bf16) {
      if (wide) NORM_PICK(residual_norm_kernel, u16, u16, 8);
      else NORM_PICK(residual_norm_kernel, u16, u16, 1);
    } else {
      if (wide) NORM_PICK(residual_norm_kernel, u16, float, 8);
      else NORM_PICK(residual_norm_kernel, u16, float, 1);
    }
  } else {
    if (wide) NORM_PICK(residual_norm_kernel, float, float, 4);
    else NORM_PICK(residual_norm_kernel, float, float, 1);
  }
  return hipGetLastError();
}

hipError_t launch_residual_norm_bwd(const ResidualNormArgs &a, hipStream_t st) {
  const int e = a.bf16 ? 2 : 4, re = a.res_bf16 ? 2 : 4, vec = 16 / e;
  const bool wide = a.dim % vec == 0 && aligned(a.x, a.x_stride, e) && aligned(a.residual, a.dim, re) &&
                    aligned(a.dy, a.dim, e) && aligned(a.dx, a.dim, e) && aligned(a.dres, a.dim, re) &&
                    (!a.dh || aligned(a.dh, a.dim, re)) && aligned(a.part, a.dim, 4) && aligned(a.w_pre, 4, 4) &&
                    (!a.w_post || aligned(a.w_post, 4, 4)) && (!a.scale || aligned(a.scale, 4, 4)) &&
                    (a.act < 0 || (aligned(a.gate, a.gate_stride, e) && aligned(a.dgate, a.dim, e)));
  const TeamPlan p = plan_rows(wide ? a.dim / vec : a.dim);
  const int grid = row_blocks(a.tokens, p, norm_bwd_blocks(a.tokens));
  TimedLaunch tl(K_NORM_BWD, st);
  if (a.bf16) {
    if (a.res_bf16) {
      if (wide) NORM_PICK(residual_norm_bwd_kernel, u16, u16, 8);
      else NORM_PICK(residual_norm_bwd_kernel, u16, u16, 1);
    } else {
      if (wide) NORM_PICK(residual_norm_bwd_kernel, u16, float, 8);
      else NORM_PICK(residual_norm_bwd_kernel, u16, float, 1);
    }
  } else {
    if (wide) NORM_PICK(residual_norm_bwd_kernel, float, float, 4);
    else NORM_PICK(residual_norm_bwd_kernel, float, float, 1);
  }
  norm_partials_kernel<<<dim3((a.dim + 63) / 64, 3), 1024, 0, st>>>(
      a.part, grid, a.dim, a.dw_pre, a.w_post ? a.dw_post : nullptr, a.scale ? a.dscale : nullptr);
  return hipGetLastError();
}

}  // namespace flare
