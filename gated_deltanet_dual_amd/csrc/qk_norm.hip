// qk_norm.hip -- the norms of queries and keys for each head with the rotary
// position in the same pass, forward and reverse mode; the forward also on the way
// into a paged cache, of the inputs' type or in 4 bits; and rows read back from a
// cache in 4 bits.
//
//   n = x r w,  r = 1 / sqrt(mean x^2 + eps)          per (token, head) row
//   y = R n:  (a, b) -> m (a cos - b sin, a sin + b cos) on the turned pairs
//
// Reverse: du = R^T dy;  dw = sum du x r;  dx = r (du w - x r^2 mean(du w x)).
//
// Memory bounds them: a row is read once into the registers of a team of lanes, a
// lane holding both members of every pair that it turns, and written once.
#include <hip/hip_runtime.h>

#include "fast_div.h"
#include "fp4.h"
#include "layer_launch.h"
#include "rotary_turn.h"
#include "vec_io.h"

namespace flare {
namespace {

struct QkNormPlan {
  int tb;     // tokens a workgroup has at a time
  int shift;  // lanes of a team: 1 << shift
  int per;    // work items of a head
  FastDiv half, q_heads, k_heads;
  int k_rows;      // into 4 bits: key rows that the workgroup's buffer holds
  FastDiv chunks;  // and a row's pieces of 8 channels
};

enum { PACKED = 0, PAGES = 1, PAGES4 = 2 };

// Where a work item's two vectors lie in a head's row and how many channels each has
// left there (n1 <= 0: there is no second one; c1 is then c0).
struct Item {
  int c0, c1, n0, n1;
  bool turned;
};
template <int VEC> __device__ __forceinline__ Item item_of(const RotaryArgs &a, int j) {
  const int turned = rotary_turned_items(a, VEC);
  Item it;
  it.turned = j < turned;
  if (it.turned && !a.interleaved) {
    it.c0 = j * VEC;
    it.c1 = a.half + it.c0;
    it.n0 = it.n1 = a.half - it.c0;
  } else {
    const int start = it.turned ? 0 : 2 * a.half, end = it.turned ? 2 * a.half : a.dim;
    it.c0 = start + 2 * (it.turned ? j : j - turned) * VEC;
    it.c1 = it.c0 + VEC;
    it.n0 = end - it.c0;
    it.n1 = end - it.c1;
    if (it.n1 <= 0) it.c1 = it.c0;
  }
  return it;
}
// A value row's item: two vectors next to each other.
template <int VEC> __device__ __forceinline__ Item copy_of(const RotaryArgs &a, int j) {
  Item it{2 * j * VEC, 2 * j * VEC + VEC, a.dim - 2 * j * VEC, a.dim - 2 * j * VEC - VEC, false};
  if (it.n1 <= 0) it.c1 = it.c0;
  return it;
}

// Both vectors of an item; zeros for what does not exist.
template <typename IO, int VEC, bool TAIL>
__device__ __forceinline__ void load_item(const IO *row, const Item &it, float (&x)[2][VEC]) {
  load_vec<IO, VEC, TAIL>(row + it.c0, it.n0, x[0]);
  load_vec<IO, VEC, TAIL>(row + it.c1, it.n1 <= 0 ? it.n0 : it.n1, x[1]);
  if (it.n1 <= 0) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[1][e] = 0.0f;
  }
}
template <typename IO, int VEC, bool TAIL>
__device__ __forceinline__ void store_item(IO *row, const Item &it, const float (&x)[2][VEC]) {
  store_vec<IO, VEC, TAIL>(row + it.c0, it.n0, x[0]);
  if (it.n1 > 0) store_vec<IO, VEC, TAIL>(row + it.c1, it.n1, x[1]);
}

// The pairs of a turned item; cf: the token's coefficients.
template <int VEC, bool TAIL, typename T, typename T2>
__device__ __forceinline__ void turn_item(const Item &it, bool interleaved, const T2 *cf, T (&x)[2][VEC]) {
  if (!it.turned) return;
  if (!interleaved) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const T2 w = cf[TAIL && e >= it.n0 ? it.c0 : it.c0 + e];
      const T u = x[0][e], v = x[1][e];
      x[0][e] = u * w.x - v * w.y;
      x[1][e] = u * w.y + v * w.x;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const T2 *c = cf + (h ? it.c1 : it.c0) / 2;
      const int n = h ? it.n1 : it.n0;
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        const T2 w = c[(TAIL || h) && e >= n ? 0 : e / 2];
        const T u = x[h][e], v = x[h][e + 1];
        x[h][e] = u * w.x - v * w.y;
        x[h][e + 1] = u * w.y + v * w.x;
      }
    }
  }
}

template <typename T> __device__ __forceinline__ T team_sum(T x, int shift) {
  for (int o = 1 << shift >> 1; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

__device__ __forceinline__ uint32_t xor_lane(uint32_t x, int o) { return __shfl_xor(x, o); }
__device__ __forceinline__ uint64_t xor_lane(uint64_t x, int o) { return __shfl_xor((unsigned long long)x, o); }

// One workgroup: `tb` tokens.  Their coefficients first, to LDS, so that a token's angles
// are formed once for all its heads; then the rows, one a team.
// Into 4 bits, keys are computed in 64 bits from their norm's sum to the rounding: a value
// next to the border of two codes, half a step apart, goes to the right one, which 32 bits
// would miss once in some 10^7 values.  They go through LDS, where groups of 32 channels
// lie together whatever pairs were turned.
template <typename IO, int VEC, bool TAIL, int NI, int OUT>
__global__ __launch_bounds__(256) void qk_norm_rotary_kernel(QkNormArgs a, QkNormPlan p) {
  using C2 = std::conditional_t<OUT == PAGES4, double2, float2>;
  extern __shared__ __align__(16) char lds[];
  C2 *coef = reinterpret_cast<C2 *>(lds);                          // [tb][half]
  int2 *place = reinterpret_cast<int2 *>(coef + p.tb * a.r.half);  // [tb] page and row in it; page < 0: nowhere
  double *keys = reinterpret_cast<double *>(place + p.tb);         // [k_rows][dim]
  const RotaryArgs &r = a.r;
  const int64_t t0 = (int64_t)blockIdx.x * p.tb;
  const int n = (int)(r.tokens - t0 < p.tb ? r.tokens - t0 : p.tb);
  for (int i = threadIdx.x; i < n * r.half; i += 256) {
    const int t = fast_div(i, p.half), j = i - t * r.half;
    if constexpr (OUT == PAGES4) {
      double s, c;
      sincospi(2.0 * turn_fraction(r.positions[t0 + t], r.freqs[j]), &s, &c);
      coef[i] = make_double2((double)r.mscale * c, (double)r.mscale * s);
    } else {
      coef[i] = turn(r.positions[t0 + t], r.freqs[j], r.mscale, 1.0f);
    }
  }
  if constexpr (OUT != PACKED) {
    if (threadIdx.x < n) {
      const int64_t slot = r.slots[t0 + threadIdx.x], all = r.num_pages * r.page;
      int2 at = make_int2(-1, 0);
      if (slot >= 0 && slot < all) {
        const int64_t pg = all <= INT32_MAX ? (int64_t)((uint32_t)slot / (uint32_t)r.page) : slot / r.page;
        at = make_int2((int)pg, (int)(slot - pg * r.page));
      }
      place[threadIdx.x] = at;
    }
  }
  __syncthreads();
  const int shift = p.shift, lane = threadIdx.x & ((1 << shift) - 1), team = threadIdx.x >> shift, teams = 256 >> shift;
  const int nq = n * r.q_heads, nk = n * r.k_heads;
  // into 4 bits: the queries and the first keys, then further keys in rounds
  for (int k0 = 0; k0 == 0 || k0 < nk; k0 += p.k_rows) {
    const int kn = OUT == PAGES4 ? (nk - k0 < p.k_rows ? nk - k0 : p.k_rows) : nk;
    const int first = k0 == 0 ? nq : 0, rows = first + kn + (OUT == PAGES ? nk : 0);
    for (int row = team; row < rows; row += teams) {
      int kind = 0, t, head;  // 0 a query, 1 a key, 2 a value
      if (row < first) {
        t = fast_div(row, p.q_heads);
        head = row - t * r.q_heads;
      } else {
        int i = row - first + k0;
        kind = 1;
        if (OUT == PAGES && i >= nk) {
          kind = 2;
          i -= nk;
        }
        t = fast_div(i, p.k_heads);
        head = i - t * r.k_heads;
      }
      const int64_t tok = t0 + t, hd = (int64_t)head * r.dim;
      const IO *src = kind == 0 ? (const IO *)r.q + tok * r.q_stride + hd
                    : kind == 1 ? (const IO *)r.k + tok * r.k_stride + hd : (const IO *)r.v + tok * r.v_stride + hd;
      IO *dst;
      if (OUT == PACKED || kind == 0) {
        dst = kind == 0 ? (IO *)r.q_out + (tok * r.q_heads + head) * r.dim : (IO *)r.k_out + (tok * r.k_heads + head) * r.dim;
      } else if constexpr (OUT == PAGES) {
        const int2 at = place[t];
        if (at.x < 0) continue;
        dst = (kind == 1 ? (IO *)r.k_cache : (IO *)r.v_cache) + (((int64_t)at.x * r.k_heads + head) * r.page + at.y) * r.dim;
      }
      Item it[NI];
      float x[NI][2][VEC];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int j = lane + (i << shift);
        it[i] = kind == 2 ? copy_of<VEC>(r, j) : item_of<VEC>(r, j);
        if (kind == 2 ? it[i].n0 > 0 : j < p.per) load_item<IO, VEC, TAIL>(src, it[i], x[i]);
        else it[i].n0 = 0;
      }
      const float *w = kind == 2 ? nullptr : a.weight[kind & 1];
      const C2 *cf = coef + t * r.half;
      // y = R (x rstd w) in T
      auto finish = [&](auto zero, auto &y) {
        using T = decltype(zero);
        if (w) {
          T ss = 0;
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if (it[i].n0 > 0) {
#pragma unroll
              for (int e = 0; e < 2 * VEC; ++e) ss += (T)x[i][e / VEC][e % VEC] * (T)x[i][e / VEC][e % VEC];
            }
          ss = team_sum(ss, shift);
          const T rstd = (T)1 / sqrt(ss / (T)r.dim + (T)a.eps);
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if (it[i].n0 > 0) {
              float wv[2][VEC];
              load_item<float, VEC, TAIL>(w, it[i], wv);
#pragma unroll
              for (int e = 0; e < 2 * VEC; ++e) y[i][e / VEC][e % VEC] = (T)x[i][e / VEC][e % VEC] * rstd * (T)wv[e / VEC][e % VEC];
            }
        } else {
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) y[i][e / VEC][e % VEC] = (T)x[i][e / VEC][e % VEC];
        }
      };
      if (OUT == PAGES4 && kind == 1) {
        double y[NI][2][VEC];
        finish(0.0, y);
        double *to = keys + (int64_t)(row - first) * r.dim;
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (it[i].n0 > 0) {
            turn_item<VEC, TAIL>(it[i], r.interleaved, cf, y[i]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              if (!TAIL || e < it[i].n0) to[it[i].c0 + e] = y[i][0][e];
              if (e < it[i].n1) to[it[i].c1 + e] = y[i][1][e];
            }
          }
      } else {
        float y[NI][2][VEC];
        finish(0.0f, y);
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (it[i].n0 > 0) {
            if (kind != 2) turn_item<VEC, TAIL>(it[i], r.interleaved, cf, y[i]);
            store_item<IO, VEC, TAIL>(dst, it[i], y[i]);
          }
      }
    }
    if constexpr (OUT != PAGES4) break;
    // the keys of the buffer and, once, the values: 8 channels a thread, four threads a group
    __syncthreads();
    const int chunks = r.dim / 8, values = k0 == 0 ? nk : 0;
    for (int i = threadIdx.x; i < (kn + values) * chunks; i += 256) {
      const int row = fast_div(i, p.chunks), c = i - row * chunks;
      const bool key = row < kn;
      const int at_row = key ? row + k0 : row - kn, t = fast_div(at_row, p.k_heads), head = at_row - t * r.k_heads;
      const int2 at = place[t];
      uint32_t codes;
      int byte;
      auto group = [&](const auto (&x)[8]) {
        auto top = abs_bits(x[0]);
#pragma unroll
        for (int e = 1; e < 8; ++e) {
          const auto b = abs_bits(x[e]);
          top = b > top ? b : top;
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          const auto b = xor_lane(top, o);
          top = b > top ? b : top;
        }
        byte = fp4_scale(top);
        codes = fp4_codes(x, byte);
      };
      if (key) {
        double x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = keys[row * r.dim + 8 * c + e];
        group(x);
      } else {
        float x[8];
        Vec<IO, 8>::load((const IO *)r.v + (t0 + t) * r.v_stride + (int64_t)head * r.dim + 8 * c, x);
        group(x);
      }
      if (at.x >= 0) {
        const Cache4 &to = key ? a.k4 : a.v4;
        const int64_t ph = (int64_t)at.x * r.k_heads + head;
        *reinterpret_cast<uint32_t *>(to.codes + ((ph * r.page + at.y) * r.dim >> 1) + 4 * c) = codes;
        if ((c & 3) == 0) to.scales[(ph * (r.dim / kFp4Group) + (c >> 2)) * r.page + at.y] = (uint8_t)byte;
      }
    }
    __syncthreads();
  }
}

// The queries' rows, then the keys', a workgroup's tokens each time: one set of weights and
// of their gradients' sums in registers, written once as a partial row, which a second
// launch adds up in a fixed order.
template <typename IO, int VEC, bool TAIL, int NI>
__global__ __launch_bounds__(256) void qk_norm_rotary_bwd_kernel(QkNormArgs a, QkNormPlan p) {
  extern __shared__ __align__(16) char lds[];
  float2 *coef = reinterpret_cast<float2 *>(lds);  // [tb][half]
  __shared__ float cols[256 * VEC];
  const RotaryArgs &r = a.r;
  const int shift = p.shift, lane = threadIdx.x & ((1 << shift) - 1), team = threadIdx.x >> shift, teams = 256 >> shift;
  Item it[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    it[i] = item_of<VEC>(r, lane + (i << shift));
    if (lane + (i << shift) >= p.per) it[i].n0 = 0;
  }
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const int heads = kind ? r.k_heads : r.q_heads;
    if (heads == 0) break;
    const FastDiv by = kind ? p.k_heads : p.q_heads;
    const float *w = a.weight[kind];
    float wv[NI][2][VEC] = {}, dw[NI][2][VEC] = {};
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (w && it[i].n0 > 0) load_item<float, VEC, TAIL>(w, it[i], wv[i]);
    for (int64_t t0 = (int64_t)blockIdx.x * p.tb; t0 < r.tokens; t0 += (int64_t)gridDim.x * p.tb) {
      const int n = (int)(r.tokens - t0 < p.tb ? r.tokens - t0 : p.tb);
      __syncthreads();
      for (int i = threadIdx.x; i < n * r.half; i += 256) {
        const int t = fast_div(i, p.half), j = i - t * r.half;
        coef[i] = turn(r.positions[t0 + t], r.freqs[j], r.mscale, -1.0f);
      }
      __syncthreads();
      for (int row = team; row < n * heads; row += teams) {
        const int t = fast_div(row, by), head = row - t * heads;
        const int64_t tok = t0 + t, hd = (int64_t)head * r.dim;
        const IO *src = (const IO *)(kind ? r.k : r.q) + tok * (kind ? r.k_stride : r.q_stride) + hd;
        const IO *dsrc = (const IO *)a.dout[kind] + tok * a.dout_stride[kind] + hd;
        IO *dst = (IO *)a.dx[kind] + (tok * heads + head) * r.dim;
        float x[NI][2][VEC], d[NI][2][VEC], ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (it[i].n0 > 0) {
            if (w) load_item<IO, VEC, TAIL>(src, it[i], x[i]);
            load_item<IO, VEC, TAIL>(dsrc, it[i], d[i]);
          }
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (it[i].n0 > 0) turn_item<VEC, TAIL>(it[i], r.interleaved, coef + t * r.half, d[i]);
        if (w) {
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if (it[i].n0 > 0) {
#pragma unroll
              for (int e = 0; e < 2 * VEC; ++e) {
                const float xe = x[i][e / VEC][e % VEC];
                ss += xe * xe;
                dot += d[i][e / VEC][e % VEC] * wv[i][e / VEC][e % VEC] * xe;
              }
            }
          for (int o = 1 << shift >> 1; o > 0; o >>= 1) {
            ss += __shfl_xor(ss, o);
            dot += __shfl_xor(dot, o);
          }
          const float rstd = 1.0f / sqrtf(ss / (float)r.dim + a.eps);
          const float mean = dot * rstd / (float)r.dim;  // of dn n
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if (it[i].n0 > 0) {
#pragma unroll
              for (int e = 0; e < 2 * VEC; ++e) {
                float &de = d[i][e / VEC][e % VEC];
                const float u = x[i][e / VEC][e % VEC] * rstd;
                dw[i][e / VEC][e % VEC] += de * u;
                de = rstd * (de * wv[i][e / VEC][e % VEC] - u * mean);
              }
            }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (it[i].n0 > 0) store_item<IO, VEC, TAIL>(dst, it[i], d[i]);
      }
    }
    if (!w) continue;
    // the teams' sums, a vector of every thread at a time
    float *out = a.part + ((int64_t)kind * gridDim.x + blockIdx.x) * r.dim;
#pragma unroll
    for (int v = 0; v < 2 * NI; ++v) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e) cols[threadIdx.x * VEC + e] = dw[v / 2][v % 2][e];
      __syncthreads();
      for (int j = threadIdx.x; j < VEC << shift; j += 256) {
        const int item = j / VEC + (v / 2 << shift), e = j % VEC;
        if (item >= p.per) continue;
        const Item at = item_of<VEC>(r, item);
        if (e >= (v % 2 ? at.n1 : at.n0)) continue;
        float s = 0.0f;
        for (int k = 0; k < teams; ++k) s += cols[(k << shift) * VEC + j];
        out[(v % 2 ? at.c1 : at.c0) + e] = s;
      }
    }
  }
}

// Rows of a cache in 4 bits as bf16 or fp32: 8 channels a thread.
template <typename IO>
__global__ __launch_bounds__(256) void cache_fp4_rows_kernel(Cache4Rows a, FastDiv chunks, FastDiv heads) {
  const int per_row = a.heads * (a.dim / 8);
  const int side = blockIdx.y;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.rows * per_row; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per_row;
    const int j = (int)(i - row * per_row), head = fast_div(j, chunks), c = j - head * (a.dim / 8);
    const int64_t slot = a.slots[row];
    uint32_t v[4] = {0, 0, 0, 0};
    if (slot >= 0 && slot < a.num_pages * a.page) {
      const int64_t pg = slot / a.page, ph = pg * a.heads + head, at = slot - pg * a.page;
      const uint32_t w = *reinterpret_cast<const uint32_t *>(a.codes[side] + ((ph * a.page + at) * a.dim >> 1) + 4 * c);
      const uint32_t s = (uint32_t)a.scales[side][(ph * (a.dim / kFp4Group) + (c >> 2)) * a.page + at] << 23;
      v[0] = fp4_pair<0>(w, s);
      v[1] = fp4_pair<1>(w, s);
      v[2] = fp4_pair<2>(w, s);
      v[3] = fp4_pair<3>(w, s);
    }
    IO *out = (IO *)a.out[side] + row * (int64_t)a.heads * a.dim + (int64_t)head * a.dim + 8 * c;
    if constexpr (sizeof(IO) == 2) {
      *reinterpret_cast<uint4 *>(out) = make_uint4(v[0], v[1], v[2], v[3]);
    } else {
      uint4 lo = make_uint4(v[0] << 16, v[0] & 0xffff0000u, v[1] << 16, v[1] & 0xffff0000u);
      uint4 hi = make_uint4(v[2] << 16, v[2] & 0xffff0000u, v[3] << 16, v[3] & 0xffff0000u);
      reinterpret_cast<uint4 *>(out)[0] = lo;
      reinterpret_cast<uint4 *>(out)[1] = hi;
    }
  }
}

QkNormPlan plan_of(const QkNormArgs &a, int vec, int tb) {
  QkNormPlan p{};
  const RotaryArgs &r = a.r;
  p.tb = tb;
  p.per = rotary_turned_items(r, vec) + rotary_copy_items(r.dim - 2 * r.half, vec);
  while (p.shift < 6 && 1 << p.shift < p.per) ++p.shift;
  p.half = make_fast_div(r.half > 0 ? r.half : 1);
  p.q_heads = make_fast_div(r.q_heads);
  p.k_heads = make_fast_div(r.k_heads > 0 ? r.k_heads : 1);
  p.k_rows = 2048 / r.dim;
  p.chunks = make_fast_div(r.dim >= 8 ? r.dim / 8 : 1);
  return p;
}

bool has_tails(const RotaryArgs &r, int vec) {
  return (r.interleaved ? 2 * r.half : r.half) % vec != 0 || (r.dim - 2 * r.half) % vec != 0 || r.dim % vec != 0;
}

template <typename IO, int VEC, int OUT> void forward(const QkNormArgs &a, hipStream_t st) {
  const RotaryArgs &r = a.r;
  const QkNormPlan p = plan_of(a, VEC, rotary_block_tokens(r));
  const int grid = (int)((r.tokens + p.tb - 1) / p.tb);
  size_t lds = (size_t)p.tb * ((OUT == PAGES4 ? sizeof(double2) : sizeof(float2)) * r.half + sizeof(int2));
  if (OUT == PAGES4) lds += (size_t)p.k_rows * r.dim * sizeof(double);
  const bool one = p.per <= 1 << p.shift;
  if (has_tails(r, VEC)) {
    if (one) qk_norm_rotary_kernel<IO, VEC, true, 1, OUT><<<grid, 256, lds, st>>>(a, p);
    else qk_norm_rotary_kernel<IO, VEC, true, 3, OUT><<<grid, 256, lds, st>>>(a, p);
  } else {
    if (one) qk_norm_rotary_kernel<IO, VEC, false, 1, OUT><<<grid, 256, lds, st>>>(a, p);
    else qk_norm_rotary_kernel<IO, VEC, false, 3, OUT><<<grid, 256, lds, st>>>(a, p);
  }
}

template <typename IO, int VEC> hipError_t reverse(QkNormArgs a, hipStream_t st) {
  const RotaryArgs &r = a.r;
  const QkNormPlan p = plan_of(a, VEC, rotary_block_tokens(r));
  int64_t grid = (r.tokens + p.tb - 1) / p.tb;
  const int64_t most = qk_norm_bwd_blocks(r.tokens);
  if (grid > most) grid = most;
  if (grid > 0) {
    const size_t lds = (size_t)p.tb * sizeof(float2) * r.half;
    const bool one = p.per <= 1 << p.shift;
    if (has_tails(r, VEC)) {
      if (one) qk_norm_rotary_bwd_kernel<IO, VEC, true, 1><<<(int)grid, 256, lds, st>>>(a, p);
      else qk_norm_rotary_bwd_kernel<IO, VEC, true, 3><<<(int)grid, 256, lds, st>>>(a, p);
    } else {
      if (one) qk_norm_rotary_bwd_kernel<IO, VEC, false, 1><<<(int)grid, 256, lds, st>>>(a, p);
      else qk_norm_rotary_bwd_kernel<IO, VEC, false, 3><<<(int)grid, 256, lds, st>>>(a, p);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.weight[0] && !a.weight[1]) return hipSuccess;
  return launch_norm_partials(a.part, (int)grid, r.dim, {a.weight[0] ? a.dweight[0] : nullptr, a.weight[1] ? a.dweight[1] : nullptr, nullptr}, st);
}

}  // namespace

hipError_t launch_qk_norm_rotary(const QkNormArgs &a, hipStream_t st) {
  if (a.r.tokens == 0) return hipSuccess;
  TimedLaunch tl(K_QK_NORM, st);
  if (a.into4) a.r.bf16 ? forward<u16, rotary_vec(true), PAGES4>(a, st) : forward<float, rotary_vec(false), PAGES4>(a, st);
  else if (a.r.slots) a.r.bf16 ? forward<u16, rotary_vec(true), PAGES>(a, st) : forward<float, rotary_vec(false), PAGES>(a, st);
  else a.r.bf16 ? forward<u16, rotary_vec(true), PACKED>(a, st) : forward<float, rotary_vec(false), PACKED>(a, st);
  return hipGetLastError();
}

hipError_t launch_qk_norm_rotary_bwd(const QkNormArgs &a, hipStream_t st) {
  TimedLaunch tl(K_QK_NORM_BWD, st);
  return a.r.bf16 ? reverse<u16, rotary_vec(true)>(a, st) : reverse<float, rotary_vec(false)>(a, st);
}

hipError_t launch_cache_fp4_rows(const Cache4Rows &a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  TimedLaunch tl(K_CACHE_FP4_ROWS, st);
  const int64_t items = a.rows * a.heads * (a.dim / 8), blocks = (items + 255) / 256;
  const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384), a.out[1] ? 2 : 1);
  const FastDiv chunks = make_fast_div(a.dim / 8), heads = make_fast_div(a.heads);
  if (a.bf16) cache_fp4_rows_kernel<u16><<<grid, 256, 0, st>>>(a, chunks, heads);
  else cache_fp4_rows_kernel<float><<<grid, 256, 0, st>>>(a, chunks, heads);
  return hipGetLastError();
}

}  // namespace flare
