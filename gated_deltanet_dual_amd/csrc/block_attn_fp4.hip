// block_attn_fp4.hip -- the serving block step of a softmax layer over a cache whose keys
// and values are held in 4 bits: as block_attn.hip,
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(s q.k_j - max),
//
// over a prefix that all requests share and the request's own keys, cut into parts that a
// second launch joins.
//
// A key's code and its group's scale make a bf16 exactly, so both products are bf16 ones
// on 16x16x32 matrix instructions, S^T = K Q^T and O^T = V^T P^T, and a lane keeps one
// query (column lane & 15) throughout.  (The instructions that take 4-bit operands
// themselves, beside queries in two fp8 halves, would need no conversion of keys, but add
// their products to 2^-14 of the largest only: scores off by 5e-6 of themselves where bf16
// products are off by 1e-8.)
//
// 4 bits make the operands small enough to need no LDS: a lane loads 32 codes of one key
// as 16 bytes, which are its share of the first product's operand (each lane group takes
// the channels that its bytes hold, the queries' are laid out alike); and for the second
// product it loads, of each of its 8 keys, the codes of D / 16 neighbouring channels,
// converts them and exchanges halves of registers in pairs, so that it holds 8 keys of one
// channel for each of D / 16 products, whose rows are every (D / 16)-th channel.  So the
// waves of a workgroup share nothing while they pass the keys: each takes every fourth
// tile of 32 keys, one tile loaded ahead in registers, and the four join at the end.
#include <hip/hip_runtime.h>

#include <type_traits>
#include <utility>

#include "attn_parts.h"
#include "fp4.h"
#include "layer_launch.h"

namespace flare {
namespace {

template <int... I, typename F> __device__ __forceinline__ void each(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F> __device__ __forceinline__ void each(F f) { each(std::make_integer_sequence<int, N>{}, f); }

// A lane's share of a tile of 32 keys in two subtiles: of each subtile's key lane & 15
// D / 8 codes and their scales; of its keys 4 grp .. 4 grp + 3 the codes of D / 16
// channels, and a byte of scale each.
template <int D> struct Tile {
  static constexpr int VW = D / 128 > 0 ? D / 128 : 1;
  uint32_t k[2][D / 32], ks[2][VW], v[8][VW], vs[2];
};

// Queries of a workgroup's rows stay in registers up to 32 of them a lane, else in LDS.
template <int D, int NQ> constexpr bool kQueriesInLds = NQ * (D / 32) > 8;
template <int D, int NQ> constexpr int kQueryBytes = kQueriesInLds<D, NQ> ? NQ * (D / 32) * 1024 : 0;

// One part: 16 NQ rows of a kv head against its keys, by four waves.
template <int D, int NQ>
__device__ __forceinline__ void part_fp4(const BlockAttnFp4Args &b, const AttnPlan &p, const Part &w, char *lds) {
  constexpr int KS = D / 32;  // steps of the first product
  constexpr int VW = Tile<D>::VW;
  constexpr int DT = D / 16;  // tiles of O; tile i's row m is channel DT m + i
  const BlockAttnArgs &a = b.a;
  const int lane = lane_id(), col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k0 = w.k0, k1 = w.k1, head = w.head;
  const uint32_t G = a.q_heads / a.kv_heads;
  const int pre_tiles = (w.pre + 31) / 32;
  const int tiles = pre_tiles + (k1 > k0 ? (k1 - k0 + 31) / 32 : 0);
  const int mine = tiles > wave ? (tiles - wave + 3) / 4 : 0;  // this wave's: wave, wave + 4, ...
  // own keys below `all` are seen by every row: the tiles below it need no mask
  const bool causal = a.causal && w.req >= 0;
  int all = causal ? w.len - (a.block - 1) : w.len;
  if (all > k1) all = k1;

  // the first key of subtile sb of tile T, no later than the last subtile that holds keys
  auto subtile = [&](int T, int sb) {
    const int end = T < pre_tiles ? w.pre : k1;
    const int j = (T < pre_tiles ? 32 * T : k0 + 32 * (T - pre_tiles)) + 16 * sb, last = (end - 1) & ~15;
    return j < last ? j : last;
  };
  // lane i holds the page of this wave's subtile i
  int page_id = 0;
  if (mine > 0) {
    const int t = (lane >> 1) < mine ? lane >> 1 : mine - 1, T = wave + 4 * t;
    page_id = (T < pre_tiles ? a.prefix_table : w.table)[subtile(T, lane & 1) >> p.page_shift];
    if (page_id < 0) page_id = 0;
    if (page_id >= a.num_pages) page_id = (int)a.num_pages - 1;
  }
  // this lane's places in a subtile
  const uint32_t k_at = col * (D / 2) + grp * (D == 64 ? 8 : 16);
  const uint32_t ks_at = (D == 64 ? grp >> 1 : grp) * (uint32_t)a.page + col;
  const uint32_t v_at = 4 * grp * (D / 2) + col * (D / 32);
  const uint32_t vs_at = (col * DT / kFp4Group) * (uint32_t)a.page + 4 * grp;
  auto load = [&](Tile<D> &x, int t) {
#pragma unroll
    for (int sb = 0; sb < 2; ++sb) {
      const int j = subtile(wave + 4 * t, sb), pg = __builtin_amdgcn_readlane(page_id, 2 * t + sb);
      const int64_t ph = (int64_t)pg * a.kv_heads + head;
      const int off = j & (a.page - 1);
      const int64_t at = ((ph << p.page_shift) + off) * (D / 2), s_at = ((ph * (D / 32)) << p.page_shift) + off;
      const uint8_t *kc = (const uint8_t *)a.k_cache + at, *vc = (const uint8_t *)a.v_cache + at;
      const uint8_t *ks = b.k_scales + s_at, *vs = b.v_scales + s_at;
      if constexpr (D == 64) {
        *reinterpret_cast<uint2 *>(x.k[sb]) = *reinterpret_cast<const uint2 *>(kc + k_at);
      } else {
#pragma unroll
        for (int h = 0; h < D / 128; ++h)
          *reinterpret_cast<uint4 *>(x.k[sb] + 4 * h) = *reinterpret_cast<const uint4 *>(kc + (k_at + 64 * h));
      }
      x.ks[sb][0] = ks[ks_at];
      if constexpr (D == 256) x.ks[sb][1] = ks[ks_at + 4 * (uint32_t)a.page];
      x.vs[sb] = *reinterpret_cast<const uint32_t *>(vs + vs_at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t *row = vc + (v_at + i * (D / 2));
        if constexpr (D == 64) x.v[4 * sb + i][0] = *reinterpret_cast<const uint16_t *>(row);
        else if constexpr (D == 128) x.v[4 * sb + i][0] = *reinterpret_cast<const uint32_t *>(row);
        else *reinterpret_cast<uint2 *>(x.v[4 * sb + i]) = *reinterpret_cast<const uint2 *>(row);
      }
    }
  };
  Tile<D> ta, tb;
  if (mine > 0) load(ta, 0);

  // the queries, whose channels are those that the keys' bytes hold, and how many own keys
  // each sees
  auto channel = [&](int s) { return D == 64 ? 16 * grp + 8 * s : 128 * (s >> 2) + 32 * grp + 8 * (s & 3); };
  auto query = [&](int n, int s) {
    const uint32_t m = w.row0 + n * 16 + col, tok = m / G;
    u32x4v z = {0, 0, 0, 0};
    if (m < w.row_end)
      z = *reinterpret_cast<const u32x4v *>((const u16 *)a.q + ((int64_t)tok * a.q_heads + head * G + (m - tok * G)) * D + channel(s));
    return z;
  };
  u32x4v *const q_lds = reinterpret_cast<u32x4v *>(lds);
  char *const join = lds + kQueryBytes<D, NQ>;
  bf16x8 q[kQueriesInLds<D, NQ> ? 1 : NQ][kQueriesInLds<D, NQ> ? 1 : KS];
  if constexpr (kQueriesInLds<D, NQ>) {
    for (int i = wave; i < NQ * KS; i += 4) q_lds[i * 64 + lane] = query(i / KS, i % KS);
    __syncthreads();
  } else {
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int s = 0; s < KS; ++s) q[n][s] = __builtin_bit_cast(bf16x8, query(n, s));
  }
  int lim[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const uint32_t tok = (w.row0 + n * 16 + col) / G;
    lim[n] = k1;
    if (causal) {
      const int seen = w.len - (a.block - 1 - ((int)tok - w.req * a.block));
      lim[n] = seen < k1 ? seen : k1;
    }
  }
  const float sc = a.scale * kLog2e;
  // how far a score may pass the kept maximum: weights up to 2^8
  const float room = fminf(8.0f / sc, 1e30f);

  floatx4 o[NQ][DT];
  float m[NQ], l[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = -INFINITY;
    l[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[n][d] = floatx4{0.f, 0.f, 0.f, 0.f};
  }

  // Tile t; x is changed.
  auto compute = [&](Tile<D> &x, int t) {
    const int T = wave + 4 * t;
    const bool own = T >= pre_tiles;
    const int kt = own ? k0 + 32 * (T - pre_tiles) : 32 * T, end = own ? k1 : w.pre;
    // some of its keys do not exist or are not seen by every row
    const bool ragged = kt + 32 > (own ? all : end);
    floatx4 s[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int sb = 0; sb < 2; ++sb) s[n][sb] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < KS; ++e) {
      bf16x8 qe[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        if constexpr (kQueriesInLds<D, NQ>) qe[n] = __builtin_bit_cast(bf16x8, q_lds[(n * KS + e) * 64 + lane]);
        else qe[n] = q[n][e];
      }
#pragma unroll
      for (int sb = 0; sb < 2; ++sb) {
        const uint32_t c = x.k[sb][e], scale = x.ks[sb][e / 4] << 23;
        const bf16x8 kf = __builtin_bit_cast(
            bf16x8, make_uint4(fp4_pair<0>(c, scale), fp4_pair<1>(c, scale), fp4_pair<2>(c, scale), fp4_pair<3>(c, scale)));
#pragma unroll
        for (int n = 0; n < NQ; ++n) mma_bf16(s[n][sb], kf, qe[n]);
      }
    }
    if (ragged) {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (kt + 16 * (e >> 2) + 4 * grp + (e & 3) >= (own ? lim[n] : end)) s[n][e >> 2][e & 3] = -INFINITY;
    }
    float top[NQ];
    bool over = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      top[n] = fmaxf(fmaxf(fmaxf(s[n][0][0], s[n][0][1]), s[n][0][2]), s[n][0][3]);
      top[n] = fmaxf(fmaxf(fmaxf(fmaxf(top[n], s[n][1][0]), s[n][1][1]), s[n][1][2]), s[n][1][3]);
      over |= top[n] > m[n] + room;
    }
    if (__any(over)) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float mn = fmaxf(m[n], xmax32(xmax16(top[n])));
        const float al = __builtin_amdgcn_exp2f((m[n] - (mn == -INFINITY ? 0.0f : mn)) * sc);
        m[n] = mn;
        l[n] *= al;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] *= al;
      }
    }
    u32x4v pb[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const float base = m[n] == -INFINITY ? 0.0f : m[n] * sc;  // a row that sees nothing yet
      float y[8], sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][e >> 2][e & 3], sc, -base));
        sum += y[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) pb[n][e] = pack_bf16x2(y[2 * e], y[2 * e + 1]);
      l[n] += sum;
    }
    if (ragged) {
      // Values of rows behind the length hold anything: 0 * NaN must not reach O.  Infinities
      // and NaN (scales of 253 and above) of keys that only some of the block's queries see
      // come to those alone.
      bool odd = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = kt + 16 * (i >> 2) + 4 * grp + (i & 3), at = 8 * (i & 3);
        const bool some = key < end && own && key >= all && (x.vs[i >> 2] >> at & 255u) >= 253;
        odd |= some;
        if (key >= end || some) {
          x.vs[i >> 2] = (x.vs[i >> 2] & ~(255u << at)) | 127u << at;
#pragma unroll
          for (int h = 0; h < VW; ++h) x.v[i][h] = 0;
        }
      }
      if (__any(odd)) {
        uint32_t *const pl = reinterpret_cast<uint32_t *>(join) + wave * NQ * 16 * 16;  // [NQ][16][32 weights]
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) pl[(n * 16 + col) * 16 + 8 * (e >> 1) + 2 * grp + (e & 1)] = pb[n][e];
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int key = all > kt ? all : kt; key < end && key < kt + 32; ++key) {
          const int pg = __builtin_amdgcn_readlane(page_id, 2 * t + ((key - kt) >> 4)), off = key & (a.page - 1);
          const int64_t ph = (int64_t)pg * a.kv_heads + head;
          float f[NQ];
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            const uint32_t two = pl[(n * 16 + col) * 16 + ((key - kt) >> 1)];
            f[n] = __uint_as_float(key & 1 ? two & 0xffff0000u : two << 16);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int ch = DT * (4 * grp + r);
            const uint32_t byte = b.v_scales[((ph * (D / 32) + ch / kFp4Group) << p.page_shift) + off];
            const uint8_t *row = (const uint8_t *)a.v_cache + ((ph << p.page_shift) + off) * (D / 2) + ch / 2;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              const uint32_t two = fp4_pair<0>(row[c], byte << 23);
#pragma unroll
              for (int n = 0; n < NQ; ++n)
                if (byte >= 253 && key < lim[n]) {
                  o[n][2 * c][r] += f[n] * __uint_as_float(two << 16);
                  o[n][2 * c + 1][r] += f[n] * __uint_as_float(two & 0xffff0000u);
                }
            }
          }
        }
      }
    }
    // the values: 8 keys a lane, their scales as a float's exponent
    uint32_t scale[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) scale[i] = ((x.vs[i >> 2] >> 8 * (i & 3)) & 255u) << 23;
    each<D / 32>([&](auto c) {
      constexpr int C = decltype(c)::value;
      uint32_t y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fp4_pair<C % 4>(x.v[i][C / 4], scale[i]);
      u32x4v even, next;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        even[i] = __builtin_amdgcn_perm(y[2 * i + 1], y[2 * i], 0x05040100u);
        next[i] = __builtin_amdgcn_perm(y[2 * i + 1], y[2 * i], 0x07060302u);
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) mma_bf16(o[n][2 * C], __builtin_bit_cast(bf16x8, even), __builtin_bit_cast(bf16x8, pb[n]));
#pragma unroll
      for (int n = 0; n < NQ; ++n) mma_bf16(o[n][2 * C + 1], __builtin_bit_cast(bf16x8, next), __builtin_bit_cast(bf16x8, pb[n]));
    });
  };
#pragma unroll 1
  for (int t = 0; t < mine; ++t) {
    if (t + 1 < mine) load(tb, t + 1);
    compute(ta, t);
    ta = tb;
  }

  // The four waves' maxima and sums, then their outputs: wave r joins the channels DT (4 grp
  // + r) .. of every row, which lie together.
  __syncthreads();
  float2 *const stat = reinterpret_cast<float2 *>(join);           // [4][NQ][16]
  float *const piece = reinterpret_cast<float *>(stat + 4 * NQ * 16);  // [wave][its 3 pieces][64][DT]
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    l[n] = xsum32(xsum16(l[n]));
    m[n] = m[n] == -INFINITY ? m[n] : m[n] * sc;
    if (grp == 0) stat[(wave * NQ + n) * 16 + col] = make_float2(m[n], l[n]);
  }
  __syncthreads();
  const int64_t rows_all = (int64_t)a.num_req * a.block * a.q_heads;
  float *const part_stat = a.part + (int64_t)(p.prefix_parts + p.own_parts) * rows_all * D;
  const bool only = p.prefix_parts + p.own_parts == 1;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float mx = -INFINITY, sum = 0.0f;
    float2 st[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      st[i] = stat[(i * NQ + n) * 16 + col];
      mx = fmaxf(mx, st[i].x);
    }
    const float base = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += st[i].y * __builtin_amdgcn_exp2f(st[i].x - base);
    const float f = __builtin_amdgcn_exp2f(m[n] - base);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (r == wave) continue;
      float *to = piece + ((wave * 3 + (r < wave ? r : r - 1)) * 64 + lane) * DT;
#pragma unroll
      for (int d = 0; d < DT; d += 4)
        *reinterpret_cast<floatx4 *>(to + d) = floatx4{o[n][d][r] * f, o[n][d + 1][r] * f, o[n][d + 2][r] * f, o[n][d + 3][r] * f};
    }
    __syncthreads();
    float out[DT];
    each<4>([&](auto r) {
      constexpr int R = decltype(r)::value;
      if (wave != R) return;
#pragma unroll
      for (int d = 0; d < DT; ++d) out[d] = o[n][d][R] * f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i == R) continue;
        const float *from = piece + ((i * 3 + (R < i ? R : R - 1)) * 64 + lane) * DT;
#pragma unroll
        for (int d = 0; d < DT; d += 4) {
          const floatx4 v = *reinterpret_cast<const floatx4 *>(from + d);
#pragma unroll
          for (int e = 0; e < 4; ++e) out[d + e] += v[e];
        }
      }
    });
    if (n + 1 < NQ) __syncthreads();
    const uint32_t mrow = w.row0 + n * 16 + col;
    if (mrow < w.row_end) {
      const uint32_t tok = mrow / G;
      const int64_t row = (int64_t)tok * a.q_heads + head * G + (mrow - tok * G);
      const int ch = DT * (4 * grp + wave);
      if (only) {
        const bool any = sum > 0.0f || sum != sum;
        const float inv = any ? 1.0f / sum : 0.0f;
        uint32_t v[DT / 2];
#pragma unroll
        for (int d = 0; d < DT / 2; ++d) v[d] = pack_bf16x2(out[2 * d] * inv, out[2 * d + 1] * inv);
        __builtin_memcpy(__builtin_assume_aligned((u16 *)a.o + row * D + ch, DT * 2 < 16 ? DT * 2 : 16), v, DT * 2);
        if (a.lse && grp == 0 && wave == 0) a.lse[row] = any ? (mx + log2f(sum)) * 0.69314718055994530942f : -INFINITY;
      } else {
        const int64_t at = (int64_t)w.out * rows_all + row;
#pragma unroll
        for (int d = 0; d < DT; d += 4)
          *reinterpret_cast<floatx4 *>(a.part + at * D + ch + d) = floatx4{out[d], out[d + 1], out[d + 2], out[d + 3]};
        if (grp == 0 && wave == 0) *reinterpret_cast<float2 *>(part_stat + at * 2) = make_float2(mx, sum);
      }
    }
  }
}

constexpr int larger(int a, int b) { return a > b ? a : b; }
template <int D, int NQ> constexpr int kLdsBytes = kQueryBytes<D, NQ> + larger(4 * NQ * 16 * 8 + 12 * 64 * (D / 16) * 4, 4 * NQ * 1024);

// NQP, NQO: row tiles of 16 for the prefix (rows of all requests) and for a request's own
// keys; WPS: waves a SIMD.
template <int D, int NQP, int NQO, int WPS>
__global__ __launch_bounds__(256, WPS) void attend_fp4_kernel(BlockAttnFp4Args b, AttnPlan p) {
  __shared__ __align__(16) char lds[larger(kLdsBytes<D, NQP>, kLdsBytes<D, NQO>)];
  Part w;
  if (!find_part<16 * NQP, 16 * NQO>(b.a, p, w)) return;
  if (NQP == NQO || w.req >= 0) part_fp4<D, NQO>(b, p, w, lds);
  else part_fp4<D, NQP>(b, p, w, lds);
}

template <int D, int NQP, int NQO, int WPS> void launch(const BlockAttnFp4Args &b, const AttnPlan &p, hipStream_t st) {
  attend_fp4_kernel<D, NQP, NQO, WPS><<<(unsigned)attn_launch_blocks(p), 256, 0, st>>>(b, p);
}

template <int D> void launch_d(const BlockAttnFp4Args &b, const AttnPlan &p, hipStream_t st) {
  if (p.prefix_tiles == 1) launch<D, 1, 1, D == 256 ? 2 : 3>(b, p, st);
  else if (p.prefix_tiles == 2 && p.own_tiles == 1) launch<D, 2, 1, 2>(b, p, st);
  else if (p.prefix_tiles == 2) launch<D, 2, 2, 2>(b, p, st);
  else if constexpr (D <= 128) {
    if (p.own_tiles == 1) launch<D, 4, 1, 2>(b, p, st);
    else if (p.own_tiles == 2) launch<D, 4, 2, 2>(b, p, st);
    else launch<D, 4, 4, 2>(b, p, st);
  }
}

}  // namespace

hipError_t launch_block_attention_fp4(const BlockAttnFp4Args &b, const AttnPlan &p, hipStream_t st) {
  TimedLaunch tl(K_BLOCK_ATTN_FP4, st);
  if (b.a.dim == 64) launch_d<64>(b, p, st);
  else if (b.a.dim == 128) launch_d<128>(b, p, st);
  else launch_d<256>(b, p, st);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_attn_join(b.a, p, st);
}

}  // namespace flare
