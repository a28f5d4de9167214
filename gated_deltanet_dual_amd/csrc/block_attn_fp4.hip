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
// Beside bf16 values the second product takes its weights in bf16: in two halves (two_halves), a
// product for each, so that outputs are off by their own rounding, 1.66e-3 of themselves in the
// mean, where weights rounded once make 2.29e-3.  It is not for nothing: 256 requests over their own
// keys take 29.9 us for 28.6, one token over 131072 keys 22.0 for 21.3, 5 rows of narrow heads
// 26.5 for 24.2, a shared prefix 125 for 104 and 56 rows at d = 256 43.7 for 41.3.
//
// Few rows (part_fp4): 4 bits make the operands small enough to need no LDS.  A lane loads
// 32 codes of one key as 16 bytes, which are its share of the first product's operand (each
// lane group takes the channels that its bytes hold, the queries' are laid out alike); and
// for the second product it loads, of each of its 8 keys, the codes of D / 16 neighbouring
// channels, converts them and exchanges halves of registers in pairs, so that it holds 8
// keys of one channel for each of D / 16 products, whose rows are every (D / 16)-th channel.
// So the waves of a workgroup share nothing while they pass the keys: each takes every
// fourth tile of 32 keys, one tile in registers while the next one is under way, and the
// four join at the end.  Memory bounds it: 256 requests x 4 tokens, 4 heads of 128, up to
// 1024 keys 30 us, 3.9 TB/s, of which the loads alone take 26.8; one token over 131072
// keys 17 us, 4.3 TB/s, and 5.4 to join.
//
// Many rows (CodesToLds): what a wave converts there would be converted again by every other
// wave with rows of the same keys; so four waves convert a tile once, into LDS, and each passes
// it with 16 or 32 rows of its own, by the loop of attn_tiles.h.  256 requests x 4 over a
// prefix of 8192: 125 us with the requests' own keys beside it, 600 TFLOP/s of the two products
// that the formula names.  No unit is full: of 280 thousand cycles the vector units are active
// in 53 %, the matrix units in 39 %, LDS in 19 %; but the two waves of a SIMD do not run the
// one beside the other (53 and 39 are nearly all), and a wave waits a third of its time for its
// turn and a quarter for loads and its fellows.  More than two do not fit: 254 registers at d =
// 128 with two row tiles.  As few rows such a prefix takes longer (attn_fp4_plan).
#include <hip/hip_runtime.h>

#include <type_traits>
#include <utility>

#include "attn_tiles.h"
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
  // lane i holds where this wave's subtile i lies: its codes in units of 16 rows, its scales
  // in units of 16 bytes
  uint32_t codes_at = 0, scales_at = 0;
  if (mine > 0) {
    const int t = (lane >> 1) < mine ? lane >> 1 : mine - 1, T = wave + 4 * t, j = subtile(T, lane & 1);
    int pg = (T < pre_tiles ? a.prefix_table : w.table)[j >> p.page_shift];
    if (pg < 0) pg = 0;
    if (pg >= a.num_pages) pg = (int)a.num_pages - 1;
    const uint32_t ph = (uint32_t)pg * a.kv_heads + head, off = (j & (a.page - 1)) >> 4;
    codes_at = (ph << (p.page_shift - 4)) + off;
    scales_at = (ph * (D / 32) << (p.page_shift - 4)) + off;
  }
  // this lane's places in a subtile
  const uint32_t k_at = col * (D / 2) + grp * (D == 64 ? 8 : 16);
  const uint32_t ks_at = (D == 64 ? grp >> 1 : grp) * (uint32_t)a.page + col;
  const uint32_t v_at = 4 * grp * (D / 2) + col * (D / 32);
  const uint32_t vs_at = (col * DT / kFp4Group) * (uint32_t)a.page + 4 * grp;
  auto load = [&](Tile<D> &x, int t) {
#pragma unroll
    for (int sb = 0; sb < 2; ++sb) {
      const int64_t at = (int64_t)(uint32_t)__builtin_amdgcn_readlane(codes_at, 2 * t + sb) * (8 * D);
      const int64_t s_at = (int64_t)(uint32_t)__builtin_amdgcn_readlane(scales_at, 2 * t + sb) * 16;
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
  static_assert(NQ * KS <= 8);  // 32 registers
  bf16x8 q[NQ][KS];
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int s = 0; s < KS; ++s) q[n][s] = __builtin_bit_cast(bf16x8, query(n, s));
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
    for (int e = 0; e < KS; ++e)
#pragma unroll
      for (int sb = 0; sb < 2; ++sb) {
        const uint32_t c = x.k[sb][e], scale = x.ks[sb][e / 4] << 23;
        const bf16x8 kf = __builtin_bit_cast(
            bf16x8, make_uint4(fp4_pair<0>(c, scale), fp4_pair<1>(c, scale), fp4_pair<2>(c, scale), fp4_pair<3>(c, scale)));
#pragma unroll
        for (int n = 0; n < NQ; ++n) mma_bf16(s[n][sb], kf, q[n][e]);
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
    u32x4v pb[NQ], rest[NQ];
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
      for (int e = 0; e < 4; ++e) {
        const uint2 w = two_halves(y[2 * e], y[2 * e + 1]);
        pb[n][e] = w.x;
        rest[n][e] = w.y;
      }
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
#pragma unroll 1
        for (int key = all > kt ? all : kt; key < end && key < kt + 32; ++key) {
          const int from = 2 * t + ((key - kt) >> 4);
          const int64_t at = (int64_t)(uint32_t)__builtin_amdgcn_readlane(codes_at, from) * 16 + (key & 15);
          const int64_t s_at = (int64_t)(uint32_t)__builtin_amdgcn_readlane(scales_at, from) * 16 + (key & 15);
          float f[NQ];
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            const int j = key - kt;
            auto weight = [&](const u32x4v &w) {
              const uint32_t lo = j & 2 ? w[1] : w[0], hi = j & 2 ? w[3] : w[2];
              const uint32_t two = __shfl(j & 16 ? hi : lo, 4 * (j & 12) + col);
              return __uint_as_float(key & 1 ? two & 0xffff0000u : two << 16);
            };
            f[n] = weight(pb[n]) + weight(rest[n]);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int ch = DT * (4 * grp + r);
            const uint32_t byte = b.v_scales[s_at + ((int64_t)(ch / kFp4Group) << p.page_shift)];
            const uint8_t *row = (const uint8_t *)a.v_cache + at * (D / 2) + ch / 2;
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
    // the values: 8 keys a lane, their scales as a float's exponent (what stands in the other
    // bits is not looked at)
    uint32_t scale[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) scale[i] = (i & 3) < 3 ? x.vs[i >> 2] << (23 - 8 * (i & 3)) : x.vs[i >> 2] >> 1;
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
#pragma unroll
      for (int n = 0; n < NQ; ++n) mma_bf16(o[n][2 * C], __builtin_bit_cast(bf16x8, even), __builtin_bit_cast(bf16x8, rest[n]));
#pragma unroll
      for (int n = 0; n < NQ; ++n) mma_bf16(o[n][2 * C + 1], __builtin_bit_cast(bf16x8, next), __builtin_bit_cast(bf16x8, rest[n]));
    });
  };
#pragma unroll 1
  for (int t = 0; t < mine; t += 2) {
    if (t + 1 < mine) load(tb, t + 1);
    compute(ta, t);
    if (t + 1 >= mine) break;
    if (t + 2 < mine) load(ta, t + 2);
    compute(tb, t + 1);
  }

  // The four waves' maxima and sums, then their outputs: wave r joins the channels DT (4 grp
  // + r) .. of every row, which lie together.
  float2 *const stat = reinterpret_cast<float2 *>(lds);            // [4][NQ][16]
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

// The tiles of the form that block_attn.hip describes, whose waves share them: a wave
// loads its 16 rows of codes into registers two tiles ahead and converts them into LDS one
// ahead.  Four lanes a row: a lane has D / 4 channels of it.  TK = 64: a wave
// has one subtile of K and of V; TK = 32: waves 0, 1 K, 2, 3 V.
template <int D, int TK> struct CodesToLds {
  static constexpr int SUBS = TK / 16, W = D / 32;  // words of codes of a lane's row, pieces in LDS
  static constexpr bool kLands = true, kHalves = true;
  const BlockAttnFp4Args &b;
  u16 *kt, *vt;
  int shift, lane, wave, sub;
  struct Codes {
    uint32_t c[W], s[D == 256 ? 2 : 1];
  } k, v;  // SUBS = 2: k alone, of whichever is this wave's
  __device__ __forceinline__ CodesToLds(const BlockAttnFp4Args &b, int shift, int lane, int wave, int sub, u16 (&kt_lds)[2][TK * D],
                                        u16 (&vt_lds)[2][TK * D])
      : b(b), kt(kt_lds[0]), vt(vt_lds[0]), shift(shift), lane(lane), wave(wave), sub(sub) {}
  // A lane's row and its quarter.  Eight neighbouring lanes write 16 bytes each to LDS at a
  // time and want eight places of 128 bytes.  Two rows' four quarters in order meet four of
  // them (d = 64, 128) or two; so the eight lanes are half quarters of four rows, every other
  // lane has its halves the other way round (d = 256) and of values, where only even places
  // change with the row, each two words.  37 requests x 7 x 16 heads of 256 over 2500 + 777
  // keys, weights rounded once: 43 us with those conflicts, half of the LDS' cycles, 37 without.
  __device__ __forceinline__ static int row_of(int lane) { return D == 64 ? lane >> 2 : (lane >> 1 & 3) | (lane >> 4 << 2); }
  __device__ __forceinline__ static int quarter_of(int lane) { return D == 64 ? lane & 3 : (lane & 1) | (lane >> 2 & 2); }
  __device__ __forceinline__ void fetch(Codes &x, const void *codes, const uint8_t *scales, int64_t ph, int row) const {
    const uint8_t *c = (const uint8_t *)codes + ((ph << shift) + row) * (D / 2);
    const uint8_t *s = scales + ((ph * (D / 32)) << shift) + row;
    const uint32_t at = row_of(lane), q = quarter_of(lane), page = 1u << shift;
    if constexpr (D == 64) {
      *reinterpret_cast<uint2 *>(x.c) = *reinterpret_cast<const uint2 *>(c + (at * (D / 2) + q * 8));
      x.s[0] = s[(q >> 1) * page + at];
    } else {
#pragma unroll
      for (int h = 0; h < D / 128; ++h) {
        const uint32_t half = D == 256 ? h ^ (q & 1) : h;
        *reinterpret_cast<uint4 *>(x.c + 4 * h) = *reinterpret_cast<const uint4 *>(c + (at * (D / 2) + q * (D / 8) + 16 * half));
        x.s[h] = s[(q * (D / 128) + half) * page + at];
      }
    }
  }
  __device__ __forceinline__ void load(int pg, int head, int row, int) {
    const int64_t ph = (int64_t)pg * b.a.kv_heads + head;
    if constexpr (SUBS == 4) {
      fetch(k, b.a.k_cache, b.k_scales, ph, row);
      fetch(v, b.a.v_cache, b.v_scales, ph, row);
    } else {
      fetch(k, wave < 2 ? b.a.k_cache : b.a.v_cache, wave < 2 ? b.k_scales : b.v_scales, ph, row);
    }
  }
  __device__ __forceinline__ void put(const Codes &x, u16 *tile, bool value) const {
    const int row = row_of(lane), q = quarter_of(lane);
    const bool turn = D == 64 ? row & 1 : value && (q & 1);
    const int piece = (value ? v_piece<D>(row, W * q) : k_piece<D>(row, W * q)) ^ (D == 256 ? 4 * (q & 1) : 0) ^ (turn ? 1 : 0);
    int to = (sub * 16 + row) * D + piece * 8;
    asm volatile("" : "+v"(to));  // formed here: the four places kept in registers throughout cost spills
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t mine = x.c[i], other = x.c[i ^ 1], c = turn ? other : mine, s = x.s[i / 4] << 23;
      *reinterpret_cast<uint4 *>(tile + (to ^ (8 * i))) =
          make_uint4(fp4_pair<0>(c, s), fp4_pair<1>(c, s), fp4_pair<2>(c, s), fp4_pair<3>(c, s));
    }
  }
  __device__ __forceinline__ void land(int buf) const {
    if constexpr (SUBS == 4) {
      put(k, kt + buf * (TK * D), false);
      put(v, vt + buf * (TK * D), true);
    } else {
      put(k, (wave < 2 ? kt : vt) + buf * (TK * D), wave >= 2);
    }
  }
};

// What this workgroup works on.  As find_part, but the row groups of a unit (kv head, part)
// of the prefix go round the XCDs: its codes are few enough for each XCD's L2 to have them
// all, and units that are no multiple of eight leave no XCD more than others.
template <int PREFIX_ROWS, int OWN_ROWS>
__device__ __forceinline__ bool find_part_fp4(const BlockAttnArgs &a, const AttnPlan &p, Part &w) {
  const uint32_t G = a.q_heads / a.kv_heads, BG = a.block * G;
  const uint32_t run = blockIdx.x / 8 / kOctets, in = blockIdx.x % (8 * kOctets), all = p.prefix_runs + p.own_runs;
  const uint32_t before = ((uint64_t)run * p.prefix_runs + all - 1) / all;  // runs of the prefix before this one
  if (((uint64_t)(run + 1) * p.prefix_runs + all - 1) / all > before) {
    const uint32_t pi = before * (8 * kOctets) + in;
    if (pi >= p.prefix_blocks) return false;
    const uint32_t unit = pi / p.prefix_groups, rg = pi % p.prefix_groups;
    const int part = (int)(unit / a.kv_heads);
    w.head = (int)(unit % a.kv_heads);
    w.row0 = rg * PREFIX_ROWS;
    w.row_end = a.num_req * BG;
    w.len = a.prefix_len;
    w.k0 = part * p.prefix_chunk;
    w.k1 = w.len - w.k0 < p.prefix_chunk ? w.len : w.k0 + p.prefix_chunk;
    w.out = part;
    w.pre = 0;
    w.req = -1;
    w.table = a.prefix_table;
    return true;
  }
  return own_part<OWN_ROWS>(a, p, (run - before) * (8 * kOctets) + in, w);
}

// What takes 16 rows a tile: a workgroup whose waves divide the keys among them (OWN = false),
// or each wave, over tiles of keys that they share (true).
template <int D> constexpr int kTileKeys = D == 256 ? 32 : 64;
template <int D, bool SHARED, int NQ> constexpr int kRows = SHARED ? 64 * NQ : 16 * NQ;

constexpr int larger(int a, int b) { return a > b ? a : b; }
template <int D, bool SHARED, int NQ>
constexpr int kLdsBytes = SHARED ? 4 * kTileKeys<D> * D * 2
                                 : 4 * NQ * 16 * 8 + 12 * 64 * (D / 16) * 4;

template <int D, bool SHARED, int NQ>
__device__ __forceinline__ void part_of(const BlockAttnFp4Args &b, const AttnPlan &p, const Part &w, char *lds) {
  if constexpr (SHARED) {
    constexpr int TK = kTileKeys<D>;
    using Tiles = u16[2][TK * D];
    const uint32_t oct = blockIdx.x / 8;
    attn_part<D, NQ, TK, CodesToLds<D, TK>>(b, p, w, w.req < 0 ? 0 : (oct + oct / 32) & 3, *reinterpret_cast<Tiles *>(lds),
                                            *reinterpret_cast<Tiles *>(lds + sizeof(Tiles)));
  } else {
    part_fp4<D, NQ>(b, p, w, lds);
  }
}

// The prefix's and the own keys' form and row tiles; WPS: waves a SIMD.
template <int D, bool PS, int NQP, bool OS, int NQO, int WPS>
__global__ __launch_bounds__(256, WPS) void attend_fp4_kernel(BlockAttnFp4Args b, AttnPlan p) {
  __shared__ __align__(16) char lds[larger(kLdsBytes<D, PS, NQP>, kLdsBytes<D, OS, NQO>)];
  Part w;
  if (!find_part_fp4<kRows<D, PS, NQP>, kRows<D, OS, NQO>>(b.a, p, w)) return;
  if ((PS == OS && NQP == NQO) || w.req >= 0) part_of<D, OS, NQO>(b, p, w, lds);
  else part_of<D, PS, NQP>(b, p, w, lds);
}

template <int D, bool PS, int NQP, bool OS, int NQO, int WPS>
hipError_t launch(const BlockAttnFp4Args &b, const AttnPlan &p, hipStream_t st) {
  attend_fp4_kernel<D, PS, NQP, OS, NQO, WPS><<<(unsigned)attn_launch_blocks(p), 256, 0, st>>>(b, p);
  return hipGetLastError();
}

template <int D> hipError_t launch_d(const BlockAttnFp4Args &b, const AttnPlan &p, const AttnForms &f, hipStream_t st) {
  constexpr int TWO = D == 256 ? 1 : 2, S = D == 64 ? 3 : 2;
  if (!f.prefix_shared) {  // nor the own keys'
    if (p.prefix_tiles == 1) return launch<D, false, 1, false, 1, D == 64 ? 4 : D == 128 ? 3 : 2>(b, p, st);
    if constexpr (D <= 128) {
      if (p.own_tiles == 1) return launch<D, false, 2, false, 1, D == 64 ? 3 : 2>(b, p, st);
      return launch<D, false, 2, false, 2, D == 64 ? 3 : 2>(b, p, st);
    }
  } else if (!f.own_shared) {
    if (p.own_tiles == 1) return launch<D, true, TWO, false, 1, S>(b, p, st);
    if constexpr (D <= 128) return launch<D, true, TWO, false, 2, S>(b, p, st);
  } else if (p.own_tiles == 2) {
    return launch<D, true, TWO, true, TWO, S>(b, p, st);
  } else {
    return launch<D, true, TWO, true, 1, S>(b, p, st);
  }
  return hipErrorInvalidConfiguration;  // no plan's
}

}  // namespace

hipError_t launch_block_attention_fp4(const BlockAttnFp4Args &b, const AttnPlan &p, const AttnForms &f, hipStream_t st) {
  TimedLaunch tl(K_BLOCK_ATTN_FP4, st);
  const hipError_t e = b.a.dim == 64 ? launch_d<64>(b, p, f, st) : b.a.dim == 128 ? launch_d<128>(b, p, f, st) : launch_d<256>(b, p, f, st);
  return e != hipSuccess ? e : launch_attn_join(b.a, p, st);
}

}  // namespace flare
