// block_attn.hip -- the serving block step of a softmax layer: the B queries of
// each request over a prefix of keys that all requests share and over the
// request's own keys, both in pages of one cache.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(s q.k_j - max),  over the prefix and own keys j together
//
// The keys are cut into parts (a range of the prefix or of a request's own
// keys); a part keeps the running maximum m, the sum l and the unnormalised
// output O of its rows, and a second launch joins the parts:
//   m = max m_i,  o = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i.
//
// Products are formed transposed, S^T = K Q^T and O^T = V^T P^T, so that a
// lane keeps one query (column lane & 15) throughout: the maximum and the sum
// are in-lane but for two lane exchanges, rescaling O is a multiplication by a
// lane's own scalar, and S^T's accumulator registers are, rounded to bf16,
// the B operand of the second product: lane group q = lane >> 4 holds the keys
// 4q..4q+3 of two 16-key subtiles, and V^T is read in that same key order by
// the LDS transpose read (16 lanes read four 32-byte row pieces, each lane
// receives one column of four rows).
#include <hip/hip_runtime.h>

#include "block_attn.h"
#include "device_common.h"
#include "layer_launch.h"

namespace flare {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr float kLog2e = 1.44269504088896340736f;

// max with lane ^ 16 and lane ^ 32
__device__ __forceinline__ float xmax16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float xmax32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Where the 16-byte piece c of row `row` of a V tile [rows][D] bf16 sits: the
// pairs of pieces that a transpose read takes from 16 rows fall on all banks.
template <int D>
__device__ __forceinline__ int v_piece(int row, int c) {
  constexpr int pairs = D / 16 < 8 ? D / 16 : 8;
  return c ^ (2 * ((D == 64 ? row >> 1 : row) & (pairs - 1)));
}

// One workgroup: NQ * 16 rows of one kv head over one part.  Its four waves
// take the part's 32-key tiles in turn, each with its own m, l and O, and are
// joined through LDS at the end.  K goes from memory straight to MFMA operand
// registers; V through a wave's own LDS tile (in-order LDS accesses of one
// wave: no barrier in the loop).  The loads of the next tile are issued as soon
// as the registers of this one are consumed.
template <int D, int NQ>
__global__ __launch_bounds__(256) void attn_rows_kernel(BlockAttnArgs a, AttnPlan p) {
  constexpr int KS = D / 32;       // MFMA steps over the head
  constexpr int DT = D / 16;       // 16-channel tiles of O
  constexpr int VL = D / 16;       // 16-byte V pieces a lane loads per tile
  constexpr int PIECES = D / 8;    // 16-byte pieces of a row
  __shared__ __align__(16) u16 lds[4][32 * D];
  __shared__ float stat[4][NQ][2][16];
  const int lane = lane_id(), wave = threadIdx.x >> 6, col = lane & 15, grp = lane >> 4;

  // which rows and keys
  int64_t id = blockIdx.x;
  const bool shared = id < p.prefix_blocks;
  const int groups = shared ? p.prefix_groups : p.own_groups;
  const int parts = shared ? p.prefix_parts : p.own_parts;
  if (!shared) id -= p.prefix_blocks;
  const int head = (int)(id % a.kv_heads);
  id /= a.kv_heads;
  const int rg = (int)(id % groups);
  id /= groups;
  const int part = (int)(id % parts);
  const int req = (int)(id / parts);  // 0 for the prefix
  const int G = a.q_heads / a.kv_heads, BG = a.block * G;
  int64_t row0, row_end;  // rows (token * G + query of the group) of this workgroup
  int len, chunk;
  const int32_t *table;
  if (shared) {
    row0 = 0;
    row_end = (int64_t)a.num_req * BG;
    len = a.prefix_len;
    chunk = p.prefix_chunk;
    table = a.prefix_table;
  } else {
    row0 = (int64_t)req * BG;
    row_end = row0 + BG;
    len = attn_own_len(a, a.seq_lens[req]);
    chunk = p.own_chunk;
    table = a.block_table + (int64_t)req * a.max_pages;
  }
  row0 += (int64_t)rg * NQ * 16;
  const int k0 = part * chunk;
  const int k1 = len - k0 < chunk ? len : k0 + chunk;
  const bool only = p.prefix_parts + p.own_parts == 1;
  // a part behind the request's length: the joining launch does not read it
  if (k0 >= k1 && !only) return;
  const int tiles = (k1 - k0 + 31) >> 5;

  // the pages of this wave's subtiles: lane i holds that of tile wave + 4 (i / 2), subtile i & 1
  int page_id = 0;
  if (k1 > k0) {
    int j = k0 + 32 * (wave + 4 * (lane >> 1)) + 16 * (lane & 1);
    const int last = (k1 - 1) & ~15;
    if (j > last) j = last;
    page_id = table[j >> p.page_shift];
    if (page_id < 0) page_id = 0;
    if (page_id >= a.num_pages) page_id = (int)a.num_pages - 1;
  }

  // the queries, and how many keys each sees
  bf16x8 q[NQ][KS];
  int lim[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int64_t m = row0 + n * 16 + col;
    lim[n] = 0;
    const bool ok = m < row_end;
    const int64_t tok = ok ? m / G : 0;
    const int g = ok ? (int)(m - tok * G) : 0;
    const u16 *src = (const u16 *)a.q + (tok * a.q_heads + head * G + g) * D;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u16x8 z = {};
      if (ok) z = *reinterpret_cast<const u16x8 *>(src + s * 32 + grp * 8);
      q[n][s] = as_bf16x8(z);
    }
    if (ok) {
      lim[n] = len;
      if (!shared && a.causal) {
        const int b = (int)(tok - (int64_t)req * a.block);
        const int seen = len - (a.block - 1 - b);
        lim[n] = seen > 0 ? seen : 0;
      }
    }
  }
  // keys below this are seen by every row
  const int all = shared || !a.causal ? len : len - (a.block - 1);
  const float sc = a.scale * kLog2e;

  floatx4 o[NQ][DT];
  float m[NQ], l[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = -INFINITY;
    l[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[n][d] = floatx4{0.f, 0.f, 0.f, 0.f};
  }

  bf16x8 kf[2][KS];
  u16x8 vr[VL];
  u16 *const vt = lds[wave];
  auto rows_of = [&](int t, int sub) -> int64_t {
    int j = k0 + 32 * t + 16 * sub;
    const int last = (k1 - 1) & ~15;
    if (j > last) j = last;
    const int pg = __builtin_amdgcn_readlane(page_id, 2 * ((t - wave) >> 2) + sub);
    return ((((int64_t)pg * a.kv_heads + head) << p.page_shift) + (j & (a.page - 1))) * D;
  };
  auto load_k = [&](int t) {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const u16 *src = (const u16 *)a.k_cache + rows_of(t, sub) + col * D + grp * 8;
#pragma unroll
      for (int s = 0; s < KS; ++s) kf[sub][s] = as_bf16x8(*reinterpret_cast<const u16x8 *>(src + s * 32));
    }
  };
  auto load_v = [&](int t) {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const u16 *src = (const u16 *)a.v_cache + rows_of(t, sub);
#pragma unroll
      for (int i = 0; i < VL / 2; ++i) {
        const int idx = i * 64 + lane;
        vr[sub * (VL / 2) + i] = *reinterpret_cast<const u16x8 *>(src + idx * 8);
      }
    }
  };
  if (wave < tiles) {
    load_k(wave);
    load_v(wave);
  }
  for (int t = wave; t < tiles; t += 4) {
    const int kt = k0 + 32 * t;
    floatx4 s[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        s[n][sub] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < KS; ++e) mma_bf16(s[n][sub], kf[sub][e], q[n][e]);
      }
    if (t + 4 < tiles) load_k(t + 4);
    // V rows behind the length hold anything: 0 * NaN must not reach O
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int idx = (i % (VL / 2)) * 64 + lane;
      const int row = (i / (VL / 2)) * 16 + idx / PIECES, c = idx % PIECES;
      u16x8 z = {};
      if (kt + row < k1) z = vr[i];
      *reinterpret_cast<u16x8 *>(vt + row * D + v_piece<D>(row, c) * 8) = z;
    }
    if (t + 4 < tiles) load_v(t + 4);

    bf16x8 pb[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int hi = lim[n] < k1 ? lim[n] : k1;
      float x[8], top = -INFINITY;
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int key = kt + 16 * sub + 4 * grp + r;
          float v = s[n][sub][r] * sc;
          if (kt + 32 > all || kt + 32 > k1) v = key < hi ? v : -INFINITY;
          x[4 * sub + r] = v;
          top = fmaxf(top, v);
        }
      top = xmax32(xmax16(top));
      const float mn = fmaxf(m[n], top);
      const float base = mn == -INFINITY ? 0.0f : mn;  // a row that sees nothing yet
      const float al = __builtin_amdgcn_exp2f(m[n] - base);
      float sum = 0.0f;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = __builtin_amdgcn_exp2f(x[e] - base);
        sum += x[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
      pb[n] = __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
      l[n] = l[n] * al + sum;
      if (__any(m[n] != mn)) {
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] *= al;
      }
      m[n] = mn;
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const int r0 = 4 * grp + (col >> 2), c = 2 * d + ((col & 3) >> 1), half = (col & 1) * 4;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vt + r0 * D + v_piece<D>(r0, c) * 8 + half));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4 *)(vt + (16 + r0) * D + v_piece<D>(16 + r0, c) * 8 + half));
      const bf16x8 vf = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
      for (int n = 0; n < NQ; ++n) mma_bf16(o[n][d], vf, pb[n]);
    }
  }

  // join the four waves: their maxima and sums, then the outputs, one query
  // tile at a time (a wave's O of 16 rows is the size of its V tile)
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    l[n] = xsum32(xsum16(l[n]));
    if (grp == 0) {
      stat[wave][n][0][col] = m[n];
      stat[wave][n][1][col] = l[n];
    }
  }
  __syncthreads();
  const int64_t rows_all = (int64_t)a.num_req * a.block * a.q_heads;
  const int out_part = shared ? part : p.prefix_parts + part;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) mx = fmaxf(mx, stat[w][n][0][col]);
    const float base = mx == -INFINITY ? 0.0f : mx;
    const float f = __builtin_amdgcn_exp2f(m[n] - base);
    float *of = reinterpret_cast<float *>(lds[wave]);
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const int c = (4 * d + grp) ^ (col & 7);  // 16-byte pieces of a row of D floats
      *reinterpret_cast<floatx4 *>(of + col * D + c * 4) = o[n][d] * f;
    }
    __syncthreads();
    // 16 rows of D floats: thread i sums piece i % (D / 4) of row i / (D / 4)
    for (int i = threadIdx.x; i < 16 * (D / 4); i += 256) {
      const int r = i / (D / 4), c = i % (D / 4);
      const int64_t mrow = row0 + n * 16 + r;
      if (mrow < row_end) {
        floatx4 sum = {0.f, 0.f, 0.f, 0.f};
        float mr = -INFINITY, lr = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          sum += *reinterpret_cast<const floatx4 *>(reinterpret_cast<const float *>(lds[w]) + r * D + (c ^ (r & 7)) * 4);
          mr = fmaxf(mr, stat[w][n][0][r]);
        }
        const float br = mr == -INFINITY ? 0.0f : mr;
#pragma unroll
        for (int w = 0; w < 4; ++w) lr += stat[w][n][1][r] * __builtin_amdgcn_exp2f(stat[w][n][0][r] - br);
        const int64_t tok = mrow / G;
        const int64_t row = tok * a.q_heads + head * G + (mrow - tok * G);
        if (only) {
          const float inv = lr > 0.0f || lr != lr ? 1.0f / lr : 0.0f;
          const uint2 w2 = make_uint2(pack_bf16x2(sum[0] * inv, sum[1] * inv), pack_bf16x2(sum[2] * inv, sum[3] * inv));
          *reinterpret_cast<uint2 *>((u16 *)a.o + row * D + c * 4) = w2;
          if (a.lse && c == 0) a.lse[row] = lr > 0.0f || lr != lr ? (mr + log2f(lr)) * 0.69314718055994530942f : -INFINITY;
        } else {
          *reinterpret_cast<floatx4 *>(a.part + ((int64_t)out_part * rows_all + row) * D + c * 4) = sum;
          if (c == 0) {
            float *ml = a.part + (int64_t)(p.prefix_parts + p.own_parts) * rows_all * D + ((int64_t)out_part * rows_all + row) * 2;
            ml[0] = mr;
            ml[1] = lr;
          }
        }
      }
    }
    __syncthreads();
  }
}

// Joins the parts of a row: D / 4 lanes a row, 16 bytes each.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(BlockAttnArgs a, AttnPlan p) {
  constexpr int L = D / 4;
  const int64_t rows = (int64_t)a.num_req * a.block * a.q_heads;
  const int64_t row = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const int c = threadIdx.x % L;
  if (row >= rows) return;
  const int req = (int)(row / ((int64_t)a.block * a.q_heads));
  const int len = attn_own_len(a, a.seq_lens[req]);
  const int parts = p.prefix_parts + (len + p.own_chunk - 1) / p.own_chunk;
  const float *ml = a.part + (int64_t)(p.prefix_parts + p.own_parts) * rows * D;
  float m = -INFINITY, l = 0.0f;
  floatx4 o = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < parts; ++i) m = fmaxf(m, ml[((int64_t)i * rows + row) * 2]);
  const float base = m == -INFINITY ? 0.0f : m;
  for (int i = 0; i < parts; ++i) {
    const float f = __builtin_amdgcn_exp2f(ml[((int64_t)i * rows + row) * 2] - base);
    l += ml[((int64_t)i * rows + row) * 2 + 1] * f;
    o += *reinterpret_cast<const floatx4 *>(a.part + ((int64_t)i * rows + row) * D + c * 4) * f;
  }
  const bool any = l > 0.0f || l != l;
  const float inv = any ? 1.0f / l : 0.0f;
  *reinterpret_cast<uint2 *>((u16 *)a.o + row * D + c * 4) =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (a.lse && c == 0) a.lse[row] = any ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

template <int D>
hipError_t launch_d(const BlockAttnArgs &a, const AttnPlan &p, hipStream_t st) {
  const int64_t blocks = p.prefix_blocks + p.own_blocks;
  if (p.tiles == 1) attn_rows_kernel<D, 1><<<(unsigned)blocks, 256, 0, st>>>(a, p);
  else attn_rows_kernel<D, 2><<<(unsigned)blocks, 256, 0, st>>>(a, p);
  if (p.prefix_parts + p.own_parts > 1) {
    const int64_t rows = (int64_t)a.num_req * a.block * a.q_heads;
    const int per = 256 / (D / 4);
    attn_join_kernel<D><<<(unsigned)((rows + per - 1) / per), 256, 0, st>>>(a, p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_attention(const BlockAttnArgs &a, hipStream_t st) {
  if (a.num_req == 0) return hipSuccess;
  const AttnPlan p = attn_plan(a);
  TimedLaunch tl(K_BLOCK_ATTN, st);
  if (a.dim == 64) return launch_d<64>(a, p, st);
  if (a.dim == 128) return launch_d<128>(a, p, st);
  return launch_d<256>(a, p, st);
}

}  // namespace flare
