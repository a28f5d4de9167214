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
//
// The weights go into the second product in bf16 (each off by at most half a step,
// 2^-8 of it, as the output's own rounding is; the matrix instructions take no wider
// ones beside bf16 values, and weights in two bf16 halves would be a third product
// beside the two): outputs of 16384 keys are off by 2.3e-3 of themselves in the mean
// where their rounding alone makes 1.7e-3.  Their sum l takes the weights unrounded;
// scores, m, l, O and the parts are fp32.
//
// What bounds it.  A prefix under many rows: the matrix instructions and the vector
// ones between them (a wave does its exponentials and its products in turn; the other
// workgroup of its CU fills some of the gaps): 16 query heads of 128, 1024 tokens x
// 8192 keys 880 TFLOP/s, 32768 keys 1025, of the 1222 that a large library product
// reaches; d = 64 868, d = 256 781.  A request's own keys: memory, 256 requests x up
// to 1024 keys, 4 heads of 128, 403 MB in 71 us, 5.7 TB/s.  Both together, side by
// side on each CU: 116 to 119 us where one after the other they take 147.  One request's
// token over 16384 keys: 8.8 us and 3.9 for the join, a launch and a few latencies
// of memory each.
#include <hip/hip_runtime.h>

#include "attn_parts.h"
#include "device_common.h"
#include "layer_launch.h"

namespace flare {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Four loads of 16 bytes of memory a lane, at base + offset bytes, straight into LDS: lane
// i's at lds + 16 i.  Written as instructions because the compiler, which cannot tell the
// tile in flight from the tile being read, waits for the one before reading the other;
// whoever reads waits for the load counter, then meets the others at a barrier.  M0, which
// names the place in LDS, is left as it was, since the compiler does not take a reserved
// register as overwritten: once for four loads (256 requests x 4 over a prefix of 8192 and
// 1024 own keys: 116.6 us, 119 once for each load, 116.1 never).  NT: own keys that no
// other workgroup reads, kept from pushing others out of the caches (256 requests' own
// 1024 keys, 4 heads of 128, from memory: 76 us where they take 85 otherwise, 32 MB 16 us
// alike; but keys that four row groups read, 64 requests x 32 tokens at d = 256: 346 us where
// they take 293).  A short prefix that every request passes goes the same way: without the
// hint for its tiles alone, 128 requests over 512 + 512 keys take 31.2 us in place of 31.7,
// over 512 + 64 keys 16.3 in place of 15.9, 256 of d = 64 over 512 + 512 20.0 in place of 20.3.
struct LdsLoad {
  const u16 *base;
  uint32_t offset, lds;
};
template <bool NT> __device__ __forceinline__ void load_lds16(const LdsLoad (&a)[4]) {
  uint32_t m0;
#define FLARE_LOAD4(HINT)                                                                                              \
  asm volatile("s_mov_b32 %0, m0\n\t"                                                                                  \
               "s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %5, %9" HINT "\n\t"                             \
               "s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %6, %10" HINT "\n\t"                            \
               "s_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %7, %11" HINT "\n\t"                            \
               "s_mov_b32 m0, %4\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %8, %12" HINT "\n\t"                            \
               "s_mov_b32 m0, %0"                                                                                      \
               : "=&s"(m0)                                                                                             \
               : "s"(a[0].lds), "s"(a[1].lds), "s"(a[2].lds), "s"(a[3].lds), "v"(a[0].offset), "v"(a[1].offset),       \
                 "v"(a[2].offset), "v"(a[3].offset), "s"(a[0].base), "s"(a[1].base), "s"(a[2].base), "s"(a[3].base)    \
               : "memory")
  if constexpr (NT) FLARE_LOAD4(" nt");
  else FLARE_LOAD4("");
#undef FLARE_LOAD4
}
// The LDS address of p, the same in all lanes.
__device__ __forceinline__ uint32_t lds_at(const u16 *p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) u16 *)p);
}
// A pointer that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const u16 *uniform(const u16 *p) {
  const uint64_t v = (uint64_t)p;
  return (const u16 *)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v) |
                       (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) << 32);
}
// Every load and LDS access of this wave done (vmcnt 0, lgkmcnt 0), then the others'.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <bool V> struct Const { static constexpr bool value = V; };

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

// One part.  The four waves hold NQ * 16 rows each and share the part's K and V
// tiles of TK keys, which memory fills straight into LDS, a tile ahead: the
// barrier that ends a tile is also the one that the next one's data waits at.
// Waves without rows (a request's few) only help to load; `turn` moves the waves
// with rows on from workgroup to workgroup, so that all SIMDs of a CU get some.
template <int D, int NQ, int TK, bool NT>
__device__ __forceinline__ void attn_part(const BlockAttnArgs &a, const AttnPlan &p, const Part &w, int turn,
                                          u16 (&kt_lds)[2][TK * D], u16 (&vt_lds)[2][TK * D]) {
  constexpr int KS = D / 32;                    // MFMA steps over the head
  constexpr int DT = D / 16;                    // 16-channel tiles of O
  constexpr int SUBS = TK / 16;                 // 16-key subtiles of a tile
  constexpr int PIECES = D / 8;                 // 16-byte pieces of a row
  constexpr int LOADS = 16 * PIECES / 64;       // 1 KiB loads of a subtile
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
  // TK = 64: a wave fills one subtile of K and of V; TK = 32: waves 0, 1 fill K, 2, 3 V.
  // A lane fetches the piece of its row that k_piece / v_piece put where it lands.
  // Row and piece of load i differ from those of load 0 by bits of i alone, so the
  // byte offset is that of load 0 with a constant's bits turned over.
  const uint32_t ky = 2 * (lane / PIECES * D + k_piece<D>(lane / PIECES, lane % PIECES) * 8);
  const uint32_t vy = 2 * (lane / PIECES * D + v_piece<D>(lane / PIECES, lane % PIECES) * 8);
  const uint32_t k_at = lds_at(&kt_lds[0][sub * 16 * D]), v_at = lds_at(&vt_lds[0][sub * 16 * D]);
  auto stage = [&](int t, int buf) {
    const int j = subtile(t), pg = __builtin_amdgcn_readlane(page_id, t);
    const int64_t at = ((((int64_t)pg * a.kv_heads + head) << p.page_shift) + (j & (a.page - 1))) * D;
    const u16 *kp = uniform((const u16 *)a.k_cache + at), *vp = uniform((const u16 *)a.v_cache + at);
    const uint32_t to = buf * (TK * D * 2);
    constexpr int RPI = 64 / PIECES;
    auto k_load = [&](int i) {
      return LdsLoad{kp, ky ^ uint32_t(2 * (i * RPI * D + k_piece<D>(i * RPI, 0) * 8)), k_at + to + i * 1024};
    };
    auto v_load = [&](int i) {
      return LdsLoad{vp, vy ^ uint32_t(2 * (i * RPI * D + v_piece<D>(i * RPI, 0) * 8)), v_at + to + i * 1024};
    };
    if constexpr (SUBS == 4) {
#pragma unroll
      for (int i = 0; i < LOADS; i += 2) load_lds16<NT>({k_load(i), v_load(i), k_load(i + 1), v_load(i + 1)});
    } else if (wave < 2) {
#pragma unroll
      for (int i = 0; i < LOADS; i += 4) load_lds16<NT>({k_load(i), k_load(i + 1), k_load(i + 2), k_load(i + 3)});
    } else {
#pragma unroll
      for (int i = 0; i < LOADS; i += 4) load_lds16<NT>({v_load(i), v_load(i + 1), v_load(i + 2), v_load(i + 3)});
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
  // V's operands of 32 keys
  auto read_v = [&](u16 *vb, int h, bf16x8 (&vf)[DT]) {
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vb + va[d % VA] + d / VA * 128 + 32 * h * D));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vb + va[d % VA] + d / VA * 128 + (32 * h + 16) * D));
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
      floatx4 s[NQ][2];
      // two subtiles in turn: 2 NQ accumulators, each product a step behind its last
#pragma unroll
      for (int e = 0; e < KS; ++e)
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
          const bf16x8 kf =
              __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4v *>(kb + ka[e % KA] + e / KA * 128 + (32 * h + 16 * sb) * D));
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            if (e == 0) s[n][sb] = floatx4{0.f, 0.f, 0.f, 0.f};
            mma_bf16(s[n][sb], kf, q[n][e]);
          }
        }
      // V's operands while the scores become weights
      bf16x8 vf[DT];
      read_v(vb, h, vf);
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
      bf16x8 pb[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float base = m[n] == -INFINITY ? 0.0f : m[n] * sc;  // a row that sees nothing yet
        float x[8], sum = 0.0f;
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][e >> 2][e & 3], sc, -base));
          sum += x[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
        pb[n] = __builtin_bit_cast(bf16x8, make_uint4(v[0], v[1], v[2], v[3]));
        l[n] += sum;
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
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int n = 0; n < NQ; ++n) mma_bf16(o[n][d], vf[d], pb[n]);
    }
  };
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
        if (t + 1 < tiles) stage(t + 1, buffer(t + 1));
        tile(0, 0, true, kt_lds[buffer(t)], vt_lds[buffer(t)], Const<false>{});
        meet();
      }
    } else if (own) {
      for (; t < whole; t += 2) {
        if (t + 1 < tiles) stage(t + 1, 1);
        tile(0, 0, true, kt_lds[0], vt_lds[0], Const<false>{});
        meet();
        if (t + 1 >= whole) {
          ++t;
          break;
        }
        if (t + 2 < tiles) stage(t + 2, 0);
        tile(0, 0, true, kt_lds[1], vt_lds[1], Const<false>{});
        meet();
      }
    }
    const int stop = own ? tiles : pre_tiles, end = own ? k1 : w.pre;
#pragma unroll 1
    for (; t < stop; ++t) {
      if (t + 1 < tiles) stage(t + 1, buffer(t + 1));
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

// NQP, NQO: row tiles of a wave for the prefix (rows of all requests) and for a
// request's own keys; NT: the own keys, and a short prefix that comes before them, in loads
// that the caches do not keep, where a request's rows are one group (measured at load_lds16).
template <int D, int NQP, int NQO, int TK, int WPS, bool NT>
__global__ __launch_bounds__(256, WPS) void attn_kernel(BlockAttnArgs a, AttnPlan p) {
  __shared__ __align__(16) u16 kt_lds[2][TK * D];
  __shared__ __align__(16) u16 vt_lds[2][TK * D];
  Part w;
  if (!find_part<64 * NQP, 64 * NQO>(a, p, w)) return;
  const uint32_t oct = blockIdx.x / 8;
  const int turn = w.req < 0 ? 0 : (oct + oct / 32) & 3;
  if (w.req < 0 || (NQP == NQO && !NT)) attn_part<D, NQP, TK, false>(a, p, w, turn, kt_lds, vt_lds);
  else attn_part<D, NQO, TK, NT>(a, p, w, turn, kt_lds, vt_lds);
}

// Joins the parts of a row: D / 4 lanes hold 16 bytes of it each.  With `split`
// above 1 that many lane groups share a row's parts and add up through LDS.  Bound by
// memory where there are many rows (16384 of 128 from 3 parts: 29 MB in 7.6 us), by
// a launch and two latencies where there are few (16 rows from 128 parts: 3.9 us).
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(BlockAttnArgs a, AttnPlan p, int split) {
  constexpr int L = D / 4;   // lanes a row
  constexpr int S = 256 / L; // lane groups of a workgroup
  __shared__ __align__(16) float acc[S][D];
  const int64_t rows = (int64_t)a.num_req * a.block * a.q_heads;
  const int c = threadIdx.x % L, sg = threadIdx.x / L, mine = sg % split;
  const int64_t row = (int64_t)blockIdx.x * (S / split) + sg / split;
  const bool live = row < rows;
  const int req = live ? (int)((uint32_t)row / (uint32_t)(a.block * a.q_heads)) : 0;
  const int len = attn_own_len(a, a.seq_lens[req]);
  const int parts = live ? p.prefix_parts + (len + p.own_chunk - 1) / p.own_chunk : 0;
  const float2 *ml = reinterpret_cast<const float2 *>(a.part + (int64_t)(p.prefix_parts + p.own_parts) * rows * D) + row;
  float m = -INFINITY, l = 0.0f;
  for (int i = c; i < parts; i += L) {
    const float2 v = ml[i * rows];
    const float mn = fmaxf(m, v.x), base = mn == -INFINITY ? 0.0f : mn;
    l = l * __builtin_amdgcn_exp2f(m - base) + v.y * __builtin_amdgcn_exp2f(v.x - base);
    m = mn;
  }
#pragma unroll
  for (int x = 1; x < L; x <<= 1) {
    const float mo = __shfl_xor(m, x), lo = __shfl_xor(l, x);
    const float mn = fmaxf(m, mo), base = mn == -INFINITY ? 0.0f : mn;
    l = l * __builtin_amdgcn_exp2f(m - base) + lo * __builtin_amdgcn_exp2f(mo - base);
    m = mn;
  }
  const float base = m == -INFINITY ? 0.0f : m;
  floatx4 o = {0.f, 0.f, 0.f, 0.f};
  const float *src = a.part + row * D + c * 4;
#pragma unroll 4
  for (int i = mine; i < parts; i += split)
    o += *reinterpret_cast<const floatx4 *>(src + i * rows * D) * __builtin_amdgcn_exp2f(ml[i * rows].x - base);
  if (split > 1) {
    *reinterpret_cast<floatx4 *>(&acc[sg][c * 4]) = o;
    __syncthreads();
    if (mine != 0) return;
    for (int i = 1; i < split; ++i) o += *reinterpret_cast<const floatx4 *>(&acc[sg + i][c * 4]);
  }
  if (!live) return;
  const bool any = l > 0.0f || l != l;
  const float inv = any ? 1.0f / l : 0.0f;
  *reinterpret_cast<uint2 *>((u16 *)a.o + row * D + c * 4) =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (a.lse && c == 0) a.lse[row] = any ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

template <int D, int NQP, int NQO, int TK, int WPS, bool NT>
hipError_t launch_d(const BlockAttnArgs &a, const AttnPlan &p, hipStream_t st) {
  attn_kernel<D, NQP, NQO, TK, WPS, NT><<<(unsigned)attn_launch_blocks(p), 256, 0, st>>>(a, p);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_attn_join(a, p, st);
}

template <int D> void join(const BlockAttnArgs &a, const AttnPlan &p, hipStream_t st) {
  const int64_t rows = (int64_t)a.num_req * a.block * a.q_heads;
  // few rows: every lane group of a workgroup on one
  constexpr int groups = 256 / (D / 4);
  const int split = rows < 512 * groups ? groups : 1;
  const int per = groups / split;
  attn_join_kernel<D><<<(unsigned)((rows + per - 1) / per), 256, 0, st>>>(a, p, split);
}

}  // namespace

hipError_t launch_attn_join(const BlockAttnArgs &a, const AttnPlan &p, hipStream_t st) {
  if (p.prefix_parts + p.own_parts <= 1) return hipSuccess;
  if (a.dim == 64) join<64>(a, p, st);
  else if (a.dim == 128) join<128>(a, p, st);
  else join<256>(a, p, st);
  return hipGetLastError();
}

hipError_t launch_block_attention(const BlockAttnArgs &a, const AttnPlan &p, hipStream_t st) {
  TimedLaunch tl(K_BLOCK_ATTN, st);
  // one tile a wave for the prefix up to d = 128: at most 64 rows in all, so one row group
  const bool alone = p.own_groups == 1;
  if (a.dim == 64) {
    if (p.own_tiles == 2) return launch_d<64, 2, 2, 64, 3, false>(a, p, st);
    if (p.prefix_tiles == 2) return alone ? launch_d<64, 2, 1, 64, 3, true>(a, p, st) : launch_d<64, 2, 1, 64, 3, false>(a, p, st);
    return launch_d<64, 1, 1, 64, 3, true>(a, p, st);
  }
  if (a.dim == 128) {
    if (p.own_tiles == 2) return launch_d<128, 2, 2, 64, 2, false>(a, p, st);
    if (p.prefix_tiles == 2) return alone ? launch_d<128, 2, 1, 64, 2, true>(a, p, st) : launch_d<128, 2, 1, 64, 2, false>(a, p, st);
    return launch_d<128, 1, 1, 64, 2, true>(a, p, st);
  }
  return alone ? launch_d<256, 1, 1, 32, 2, true>(a, p, st) : launch_d<256, 1, 1, 32, 2, false>(a, p, st);
}

}  // namespace flare
