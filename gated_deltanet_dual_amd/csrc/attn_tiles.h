// attn_tiles.h -- a part of a block attention whose key and value tiles lie in LDS, shared by
// the workgroup's four waves.
#pragma once

#include "attn_parts.h"

namespace flare {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Every load and LDS access of this wave done (vmcnt 0, lgkmcnt 0), then the others'.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <bool V> struct Const { static constexpr bool value = V; };
template <int A, int B> struct Range { static constexpr int from = A, to = B; };

// Where the 16-byte piece c of row `row` of a V tile [rows][D] bf16 sits: the
// pairs of pieces that a transpose read takes from 16 rows fall on all banks.
template <int D>
__device__ __forceinline__ int v_piece(int row, int c) {
  constexpr int pairs = D / 16 < 8 ? D / 16 : 8;
  return c ^ (2 * ((D == 64 ? row >> 1 : row) & (pairs - 1)));
}

// Where the 16-byte piece c of row `row` of a K tile [rows][D] bf16 sits: the 16
// rows whose same piece one operand read takes fall on all banks.
template <int D>
__device__ __forceinline__ int k_piece(int row, int c) {
  constexpr int pieces = D / 8 < 16 ? D / 8 : 16;
  return c ^ ((D == 64 ? row >> 1 : row) & (pieces - 1));
}

__device__ __forceinline__ const BlockAttnArgs &attn_args(const BlockAttnArgs &a) { return a; }
__device__ __forceinline__ const BlockAttnArgs &attn_args(const BlockAttnFp4Args &b) { return b.a; }

// One part.  The four waves hold NQ * 16 rows each and share the part's K and V
// tiles of TK keys, which `from` fetches a tile ahead, into LDS: the barrier that
// ends a tile is also the one that the next one's data waits at.
// Waves without rows (a request's few) only help to load; `turn` moves the waves
// with rows on from workgroup to workgroup, so that all SIMDs of a CU get some.
// from.load(page, head, row in it, buffer) begins to fetch this wave's 16 rows of a tile.
// Where From::kLands they come to registers, a tile earlier, and from.land(buffer) writes
// them to LDS.  Where From::kHalves the weights go into the second product in two halves
// (two_halves), which leaves fewer registers: half of the values' operands are read late, and
// places in a tile are formed where they are used.
template <int D, int NQ, int TK, typename From, typename Args>
__device__ __forceinline__ void attn_part(const Args &args, const AttnPlan &p, const Part &w, int turn,
                                          u16 (&kt_lds)[2][TK * D], u16 (&vt_lds)[2][TK * D]) {
  const BlockAttnArgs &a = attn_args(args);
  constexpr int KS = D / 32;                    // MFMA steps over the head
  constexpr int DT = D / 16;                    // 16-channel tiles of O
  constexpr int SUBS = TK / 16;                 // 16-key subtiles of a tile
  constexpr int PIECES = D / 8;                 // 16-byte pieces of a row
  const int lane = lane_id(), col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k0 = w.k0, k1 = w.k1, head = w.head;
  const uint32_t G = a.q_heads / a.kv_heads;
  const uint32_t row0 = w.row0 + ((wave + turn) & 3) * (NQ * 16);
  const bool live = row0 < w.row_end;
  const int pre_tiles = (w.pre + TK - 1) / TK;
  const int tiles = pre_tiles + (k1 > k0 ? (k1 - k0 + TK - 1) / TK : 0);
  // own keys below `all` are seen by every row: the tiles below it need no mask
  const bool causal = a.causal && w.req >= 0;
  int all = causal ? w.len - (a.block - 1) : w.len;
  if (all > k1) all = k1;

  // the first key of this wave's subtile of tile t, no later than the last subtile
  // that holds keys: of the prefix for the first pre_tiles, else of the own keys
  const int sub = wave % SUBS;
  auto subtile = [&](int t) {
    const int end = t < pre_tiles ? w.pre : k1;
    const int j = (t < pre_tiles ? TK * t : k0 + TK * (t - pre_tiles)) + 16 * sub, last = (end - 1) & ~15;
    return j < last ? j : last;
  };
  // lane i holds the page of tile i's
  int page_id = 0;
  if (tiles > 0) {
    const int t = lane < tiles ? lane : tiles - 1;
    page_id = (t < pre_tiles ? a.prefix_table : w.table)[subtile(t) >> p.page_shift];
    if (page_id < 0) page_id = 0;
    if (page_id >= a.num_pages) page_id = (int)a.num_pages - 1;
  }
  From from(args, p.page_shift, lane, wave, sub, kt_lds, vt_lds);
  auto stage = [&](int t, int buf) {
    const int j = subtile(t);
    from.load(__builtin_amdgcn_readlane(page_id, t), head, j & (a.page - 1), buf);
  };
  // tile t, if there is one, on its way to its buffer before the tile at hand is passed
  auto ahead = [&](int t, int buf) {
    if constexpr (From::kLands) {
      if (t < tiles) from.land(buf);
      if (t + 1 < tiles) stage(t + 1, buf);
    } else if (t < tiles) {
      stage(t, buf);
    }
  };
  // tile t's buffer: the own keys' first is buffer 0
  auto buffer = [&](int t) { return (t + pre_tiles) & 1; };
  if (tiles > 0) stage(0, buffer(0));

  // the queries, and in the last tiles of a request how many keys each sees
  bf16x8 q[NQ][KS];
  int lim[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const uint32_t m = row0 + n * 16 + col;
    const uint32_t tok = m / G;
    const u16 *src = (const u16 *)a.q + ((int64_t)tok * a.q_heads + head * G + (m - tok * G)) * D + grp * 8;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4v z = {0, 0, 0, 0};
      if (m < w.row_end) z = *reinterpret_cast<const u32x4v *>(src + s * 32);
      q[n][s] = __builtin_bit_cast(bf16x8, z);
    }
    lim[n] = k1;
    if (causal) {
      const int seen = w.len - (a.block - 1 - ((int)tok - w.req * a.block));
      lim[n] = seen < k1 ? seen : k1;
    }
  }
  const float sc = a.scale * kLog2e;
  // how far a score may pass the kept maximum: weights up to 2^8 (finite, so that
  // the first score passes -inf + room)
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
  // this lane's places in a tile: K operand step e, V channel tile d; rows
  // further down by multiples of 16 are constant offsets from them, and so are
  // steps and channel tiles beyond the 256 bytes in which the pieces change places
  constexpr int KA = KS < 4 ? KS : 4, VA = DT < 8 ? DT : 8;
  int ka[KA], va[VA];
#pragma unroll
  for (int e = 0; e < KA; ++e) ka[e] = col * D + k_piece<D>(col, 4 * e + grp) * 8;
#pragma unroll
  for (int d = 0; d < VA; ++d) {
    const int r = 4 * grp + (col >> 2);
    va[d] = r * D + v_piece<D>(r, 2 * d + ((col & 3) >> 1)) * 8 + (col & 1) * 4;
  }
  // places differ from the first by bits of e or d alone
  int k_first = ka[0], v_first = va[0];
  auto k_at = [&](int e) { return From::kHalves ? k_first ^ (32 * e) : ka[e]; };
  auto v_at = [&](int d) { return From::kHalves ? v_first ^ (16 * d) : va[d]; };
  // V's operands of 32 keys, of some of the channel tiles
  auto read_v = [&](u16 *vb, int h, bf16x8 (&vf)[DT], auto tiles) {
#pragma unroll
    for (int d = tiles.from; d < tiles.to; ++d) {
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vb + v_at(d % VA) + d / VA * 128 + 32 * h * D));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vb + v_at(d % VA) + d / VA * 128 + (32 * h + 16) * D));
      vf[d] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  };
  // keys kt .. of a tile, of which those below `end` exist; ragged: not all of them
  // are seen by every row
  auto tile = [&](int kt, int end, bool own, const u16 *kb, u16 *vb, auto ragged) {
    bool odd = false;
    if constexpr (ragged.value) {
      // V rows behind the length hold anything: 0 * NaN must not reach O.  Rows that
      // only some of the block's queries see are looked through for infinities and NaN.
      if (kt + TK > end || (own && kt + TK > all)) {
        bool mine = false;
        for (int i = threadIdx.x; i < TK * PIECES; i += 256) {
          const int key = kt + i / PIECES;
          if (key >= end) {
            *reinterpret_cast<u32x4v *>(vb + 8 * i) = u32x4v{0, 0, 0, 0};
          } else if (own && key >= all) {
            const u32x4v v = *reinterpret_cast<const u32x4v *>(vb + 8 * i);
#pragma unroll
            for (int e = 0; e < 4; ++e) mine |= (v[e] & 0x7f80u) == 0x7f80u || (v[e] & 0x7f800000u) == 0x7f800000u;
          }
        }
        odd = __syncthreads_or(mine);
      }
    }
    if (!live) return;
#pragma unroll
    for (int h = 0; h < TK / 32; ++h) {
      if constexpr (From::kHalves) asm volatile("" : "+v"(k_first), "+v"(v_first));
      floatx4 s[NQ][2];
      // two subtiles in turn: 2 NQ accumulators, each product a step behind its last
#pragma unroll
      for (int e = 0; e < KS; ++e)
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
          const bf16x8 kf =
              __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4v *>(kb + k_at(e % KA) + e / KA * 128 + (32 * h + 16 * sb) * D));
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            if (e == 0) s[n][sb] = floatx4{0.f, 0.f, 0.f, 0.f};
            mma_bf16(s[n][sb], kf, q[n][e]);
          }
        }
      // V's operands while the scores become weights
      bf16x8 vf[DT];
      constexpr int kEarly = From::kHalves ? DT / 2 : DT;
      read_v(vb, h, vf, Range<0, kEarly>());
      float top[NQ];
      bool over = false;
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        if constexpr (ragged.value) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (kt + 32 * h + 16 * (e >> 2) + 4 * grp + (e & 3) >= (own ? lim[n] : end)) s[n][e >> 2][e & 3] = -INFINITY;
        }
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
      bf16x8 pb[NQ], rest[From::kHalves ? NQ : 1];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float base = m[n] == -INFINITY ? 0.0f : m[n] * sc;  // a row that sees nothing yet
        float x[8], sum = 0.0f;
        uint32_t v[4], r[4];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][e >> 2][e & 3], sc, -base));
          sum += x[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (From::kHalves) {
            const uint2 w = two_halves(x[2 * e], x[2 * e + 1]);
            v[e] = w.x;
            r[e] = w.y;
          } else {
            v[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
          }
        }
        if constexpr (From::kHalves) rest[n] = __builtin_bit_cast(bf16x8, make_uint4(r[0], r[1], r[2], r[3]));
        pb[n] = __builtin_bit_cast(bf16x8, make_uint4(v[0], v[1], v[2], v[3]));
        l[n] += sum;
      }
      if constexpr (From::kHalves) {
        asm volatile("" ::: "memory");  // not before the weights
        read_v(vb, h, vf, Range<kEarly, DT>());
      }
      if constexpr (ragged.value) {
        if (odd) {
          // infinities and NaN out of the product, where the weight 0 of a query that
          // does not see their key would spread them, and added to those that do
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            u32x4v v = __builtin_bit_cast(u32x4v, vf[d]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((v[e] & 0x7f80u) == 0x7f80u) v[e] &= 0xffff0000u;
              if ((v[e] & 0x7f800000u) == 0x7f800000u) v[e] &= 0xffffu;
            }
            vf[d] = __builtin_bit_cast(bf16x8, v);
          }
#pragma unroll 1
          for (int j = 0; j < 32; ++j) {
            const int row = 32 * h + j;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              const uint2 v = *reinterpret_cast<const uint2 *>(vb + row * D + v_piece<D>(row, 2 * d + (grp >> 1)) * 8 + (grp & 1) * 4);
              const float f[4] = {__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                                  __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u)};
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                  o[n][d][r] += (__float_as_uint(f[r]) & 0x7f800000u) == 0x7f800000u && kt + row < lim[n] ? f[r] : 0.0f;
            }
          }
        }
      }
#pragma unroll
      for (int c = 0; c < DT; c += kEarly) {
#pragma unroll
        for (int d = c; d < c + kEarly; ++d)
#pragma unroll
          for (int n = 0; n < NQ; ++n) mma_bf16(o[n][d], vf[d], pb[n]);
        if constexpr (From::kHalves) {
#pragma unroll
          for (int d = c; d < c + kEarly; ++d)
#pragma unroll
            for (int n = 0; n < NQ; ++n) mma_bf16(o[n][d], vf[d], rest[n]);
        }
      }
    }
  };
  if constexpr (From::kLands) {
    if (tiles > 0) from.land(buffer(0));
    if (tiles > 1) stage(1, 0);
  }
  meet();
  // The prefix's tiles (with masks: one loop for all that may need them), then the
  // own keys that every row sees, two tiles a pass so that the buffers are
  // constants (at d = 256 one, with the buffer computed: two would spill registers),
  // then the last ones with masks.
  const int whole = pre_tiles + (all > k0 ? (all - k0) / TK : 0);
  int t = 0;
#pragma unroll 1
  for (int own = pre_tiles > 0 ? 0 : 1; own < 2; ++own) {
    if (own && D == 256) {
#pragma unroll 1
      for (; t < whole; ++t) {
        ahead(t + 1, buffer(t + 1));
        tile(0, 0, true, kt_lds[buffer(t)], vt_lds[buffer(t)], Const<false>{});
        meet();
      }
    } else if (own) {
      for (; t < whole; t += 2) {
        ahead(t + 1, 1);
        tile(0, 0, true, kt_lds[0], vt_lds[0], Const<false>{});
        meet();
        if (t + 1 >= whole) {
          ++t;
          break;
        }
        ahead(t + 2, 0);
        tile(0, 0, true, kt_lds[1], vt_lds[1], Const<false>{});
        meet();
      }
    }
    const int stop = own ? tiles : pre_tiles, end = own ? k1 : w.pre;
#pragma unroll 1
    for (; t < stop; ++t) {
      ahead(t + 1, buffer(t + 1));
      tile(own ? k0 + TK * (t - pre_tiles) : TK * t, end, own, kt_lds[buffer(t)], vt_lds[buffer(t)], Const<true>{});
      meet();
    }
  }

  const int64_t rows_all = (int64_t)a.num_req * a.block * a.q_heads;
  float *stat = a.part + (int64_t)(p.prefix_parts + p.own_parts) * rows_all * D;
  const bool only = p.prefix_parts + p.own_parts == 1;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const uint32_t mrow = row0 + n * 16 + col;
    l[n] = xsum32(xsum16(l[n]));
    if (mrow < w.row_end) {
      const uint32_t tok = mrow / G;
      const int64_t row = (int64_t)tok * a.q_heads + head * G + (mrow - tok * G);
      const float mx = m[n] == -INFINITY ? m[n] : m[n] * sc;
      if (only) {
        const bool any = l[n] > 0.0f || l[n] != l[n];
        const float inv = any ? 1.0f / l[n] : 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
          *reinterpret_cast<uint2 *>((u16 *)a.o + row * D + 16 * d + 4 * grp) =
              make_uint2(pack_bf16x2(o[n][d][0] * inv, o[n][d][1] * inv), pack_bf16x2(o[n][d][2] * inv, o[n][d][3] * inv));
        if (a.lse && grp == 0) a.lse[row] = any ? (mx + log2f(l[n])) * 0.69314718055994530942f : -INFINITY;
      } else {
        const int64_t at = (int64_t)w.out * rows_all + row;
#pragma unroll
        for (int d = 0; d < DT; ++d) *reinterpret_cast<floatx4 *>(a.part + at * D + 16 * d + 4 * grp) = o[n][d];
        if (grp == 0) *reinterpret_cast<float2 *>(stat + at * 2) = make_float2(mx, l[n]);
      }
    }
  }
}

}  // namespace flare
