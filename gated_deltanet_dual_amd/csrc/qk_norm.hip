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
// lane holding both members of every pair that it turns, and written once.  What they
// reach hangs on loads under way: the next row's vectors stay as they came (converting
// them would wait for them) while a row is finished, so each half of the loop has its
// own; weights and coefficients come from LDS, for a load from memory that is waited for
// waits for all before it as well.  32768 tokens of 16 query and 4 key heads of 128 in
// bf16, the kernels alone: forward 58 us (5.7 TB/s of x and y; 92 with loads and weights
// in turn), reverse 106 us (4.8 TB/s of x, dy and dx; 167), where its instructions, some 35
// a channel, weigh as much, and 4.2 us for the weights' partial rows.  fp32, 16384 tokens:
// 56 and 106 us.  Short vectors cost: heads of 80 in bf16, 50 channels turned as halves, 70
// and 105 us (3.0 TB/s).  Below some 2000 tokens the chain of a workgroup's loads bounds it:
// 1024 tokens 5.3 and 9.5 us.  Into a cache of the rows' own type 16384 tokens take 44 us in
// bf16 and 81 in fp32 (4.5 and 5.0 TB/s).
#include <hip/hip_runtime.h>

#include "fast_div.h"
#include "fp4.h"
#include "layer_launch.h"
#include "rotary_turn.h"
#include "vec_io.h"

namespace flare {
namespace {

struct QkNormPlan {
  QkNormTiles t;
  int wave_keys;  // into 4 bits: LDS values of the rows that a wave has at a time
  float inv_dim;
  FastDiv half, q_heads, k_heads;
  FastDiv chunks, v_items;  // into 4 bits: a row's pieces of 8 channels, a token's values' pieces
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

// VEC channels of a row as they lie in memory, so that they can be under way while another
// row is finished: a conversion would have to wait for them.  A vector that would pass the
// row's end is read from the row's last VEC channels and shifted.
template <typename IO, int VEC> struct Raw {
  uint32_t w[VEC * sizeof(IO) / 4];
};
template <typename IO, int VEC, bool TAIL>
__device__ __forceinline__ void load_raw(const IO *row, int c, int dim, Raw<IO, VEC> &to) {
  if (!TAIL || dim >= VEC) {
    __builtin_memcpy(to.w, row + (TAIL && c > dim - VEC ? dim - VEC : c), sizeof(to.w));
  } else {
    IO x[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = row[c + e < dim ? c + e : 0];
    __builtin_memcpy(to.w, x, sizeof(to.w));
  }
}
// Which bits of a vector's words are of its n channels.
template <typename IO, int VEC> __device__ __forceinline__ Raw<IO, VEC> mask_of(int n) {
  Raw<IO, VEC> m;
#pragma unroll
  for (int i = 0; i < (int)(VEC * sizeof(IO) / 4); ++i) {
    if constexpr (sizeof(IO) == 2) m.w[i] = n > 2 * i + 1 ? ~0u : n > 2 * i ? 0xffffu : 0u;
    else m.w[i] = n > i ? ~0u : 0u;
  }
  return m;
}
// The channels that exist, then zeros.
template <typename IO, int VEC, bool TAIL>
__device__ __forceinline__ void unpack(const Raw<IO, VEC> &from, const Raw<IO, VEC> &mask, int c, int n, int dim, float (&x)[VEC]) {
  constexpr int kWords = VEC * sizeof(IO) / 4;
  uint32_t w[kWords];
  if constexpr (TAIL) {
    static_assert(VEC == 4);
    const int by = dim >= VEC && c > dim - VEC ? c - (dim - VEC) : 0;
    if constexpr (sizeof(IO) == 2) {
      const uint64_t v = (from.w[0] | (uint64_t)from.w[1] << 32) >> (16 * by);
      w[0] = (uint32_t)v;
      w[1] = (uint32_t)(v >> 32);
    } else {
      w[0] = by & 1 ? from.w[1] : from.w[0];
      w[1] = by & 1 ? from.w[2] : from.w[1];
      w[2] = by & 1 ? from.w[3] : from.w[2];
      w[0] = by & 2 ? (by & 1 ? from.w[3] : from.w[2]) : w[0];
      w[1] = by & 2 ? from.w[3] : w[1];
      w[3] = from.w[3];
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] &= mask.w[i];
  } else {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = n > 0 ? from.w[i] : 0;
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    if constexpr (sizeof(IO) == 2) x[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    else x[e] = __uint_as_float(w[e]);
  }
}
template <typename IO, int VEC, bool TAIL>
__device__ __forceinline__ void load_item(const IO *row, const Item &it, int dim, Raw<IO, VEC> (&to)[2]) {
  load_raw<IO, VEC, TAIL>(row, it.c0, dim, to[0]);
  load_raw<IO, VEC, TAIL>(row, it.c1, dim, to[1]);
}
template <typename IO, int VEC, bool TAIL>
__device__ __forceinline__ void store_item(IO *row, const Item &it, const float (&x)[2][VEC]) {
  store_vec<IO, VEC, TAIL>(row + it.c0, it.n0, x[0]);
  if (it.n1 > 0) store_vec<IO, VEC, TAIL>(row + it.c1, it.n1, x[1]);
}

// N values at p, ALIGNED to 16 bytes or not.  Of a short vector those behind its own are
// read too and meet zeros: more of the head's weights, one of which that is not finite makes
// the row's sums so by itself, or zeros.
template <int N, bool ALIGNED, typename T> __device__ __forceinline__ void read_lds(const T *p, T (&x)[N]) {
  if constexpr (ALIGNED) {
    static_assert(N * sizeof(T) % 16 == 0);
    uint4 v[N * sizeof(T) / 16];
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) v[i] = reinterpret_cast<const uint4 *>(p)[i];
    __builtin_memcpy(x, v, sizeof(x));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = p[i];
  }
}

// a b + c, rounded once: named, so that every form of a kernel rounds alike.
__device__ __forceinline__ float fused(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ __forceinline__ double fused(double a, double b, double c) { return __builtin_fma(a, b, c); }

// The pairs of a turned item; cf: the token's coefficients.
template <int VEC, bool TAIL, typename T, typename T2>
__device__ __forceinline__ void turn_item(const Item &it, bool interleaved, const T2 *cf, T (&x)[2][VEC]) {
  if (!it.turned) return;
  if (!interleaved) {
    T2 w[VEC];
    read_lds<VEC, !TAIL>(cf + it.c0, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const T u = x[0][e], v = x[1][e];
      x[0][e] = fused(u, w[e].x, -(v * w[e].y));
      x[1][e] = fused(u, w[e].y, v * w[e].x);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      T2 w[VEC / 2];
      read_lds<VEC / 2, !TAIL>(cf + (h ? it.c1 : it.c0) / 2, w);
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        const T u = x[h][e], v = x[h][e + 1];
        x[h][e] = fused(u, w[e / 2].x, -(v * w[e / 2].y));
        x[h][e + 1] = fused(u, w[e / 2].y, v * w[e / 2].x);
      }
    }
    asm volatile("");  // keeps the two branches' last stores apart: joined, x could not stay in registers
  }
}

// x of another lane: xor 1 and 2 within four lanes, and, where the four (eight) lanes hold the
// same, the other four of eight (eight of sixteen).
template <int CTRL> __device__ __forceinline__ float other(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
template <int CTRL> __device__ __forceinline__ double other(double x) {
  const int2 v = __builtin_bit_cast(int2, x);
  return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_mov_dpp(v.x, CTRL, 0xf, 0xf, true),
                                              __builtin_amdgcn_mov_dpp(v.y, CTRL, 0xf, 0xf, true)));
}
template <typename T> __device__ __forceinline__ T team_sum(T x, int shift) {
  if (shift > 0) x += other<0xb1>(x);   // quad_perm 1 0 3 2
  if (shift > 1) x += other<0x4e>(x);   // quad_perm 2 3 0 1
  if (shift > 2) x += other<0x141>(x);  // row_half_mirror
  if (shift > 3) x += other<0x140>(x);  // row_mirror
  if (shift > 4) x += __shfl_xor(x, 16);
  if (shift > 5) x += __shfl_xor(x, 32);
  return x;
}

// A token's page and row in it; page < 0: nowhere.
__device__ __forceinline__ int2 place_of(const RotaryArgs &r, int64_t tok) {
  const int64_t slot = r.slots[tok], all = r.num_pages * r.page;
  if (slot < 0 || slot >= all) return make_int2(-1, 0);
  const int64_t pg = all <= INT32_MAX ? (int64_t)((uint32_t)slot / (uint32_t)r.page) : slot / r.page;
  return make_int2((int)pg, (int)(slot - pg * r.page));
}

// Eight channels of a row into 4 bits: four neighbouring lanes hold a group of 32.
template <typename T>
__device__ __forceinline__ void store_fp4(const Cache4 &to, const RotaryArgs &r, int2 at, int head, int chunk, const T (&x)[8]) {
  uint32_t top = abs_bits(x[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    const uint32_t b = abs_bits(x[e]);
    top = b > top ? b : top;
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const uint32_t b = __shfl_xor(top, o);
    top = b > top ? b : top;
  }
  const int byte = fp4_scale<T>(top);
  const uint32_t codes = fp4_codes(x, byte);
  if (at.x < 0) return;
  const int64_t ph = (int64_t)at.x * r.k_heads + head;
  *reinterpret_cast<uint32_t *>(to.codes + ((ph * r.page + at.y) * r.dim >> 1) + 4 * chunk) = codes;
  if ((chunk & 3) == 0) to.scales[(ph * (r.dim / kFp4Group) + (chunk >> 2)) * r.page + at.y] = (uint8_t)byte;
}

// 1 / sqrt(mean x^2 + eps), a row's.
template <typename T, int NI, int VEC>
__device__ __forceinline__ T rstd_of(const float (&x)[NI][2][VEC], float inv_dim, int dim, float eps, int shift) {
  T ss = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fused((T)x[i][h][e], (T)x[i][h][e], ss);
  ss = team_sum(ss, shift);
  if constexpr (sizeof(T) == 8) return (T)1 / sqrt(ss / (T)dim + (T)eps);
  else return rsqrtf(fused(ss, inv_dim, eps));
}
// y = x rstd w, not yet turned.  w: the weights in LDS.
template <typename T, int VEC, bool TAIL, int NI>
__device__ __forceinline__ void weigh_row(const float (&x)[NI][2][VEC], T rstd, const float *w, const Item (&it)[NI], T (&y)[NI][2][VEC]) {
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float wv[VEC];
      read_lds<VEC, !TAIL>(w + (h ? it[i].c1 : it[i].c0), wv);
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[i][h][e] = (T)x[i][h][e] * rstd * (T)wv[e];
    }
}

template <typename IO, int VEC, bool TAIL, int NI>
__device__ __forceinline__ void load_row(const IO *row, const Item (&it)[NI], int dim, Raw<IO, VEC> (&to)[NI][2]) {
#pragma unroll
  for (int i = 0; i < NI; ++i) load_item<IO, VEC, TAIL>(row, it[i], dim, to[i]);
}
template <typename IO, int VEC, bool TAIL, int NI>
__device__ __forceinline__ void unpack_row(const Raw<IO, VEC> (&from)[NI][2], const Item (&it)[NI], int dim, float (&x)[NI][2][VEC]) {
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    unpack<IO, VEC, TAIL>(from[i][0], mask_of<IO, VEC>(it[i].n0), it[i].c0, it[i].n0, dim, x[i][0]);
    unpack<IO, VEC, TAIL>(from[i][1], mask_of<IO, VEC>(it[i].n1), it[i].c1, it[i].n1, dim, x[i][1]);
  }
}
// This lane's items of a head; one that it does not have has no channels.
template <int VEC, int NI> __device__ __forceinline__ void items_of(int per, int shift, const RotaryArgs &r, int lane, Item (&it)[NI]) {
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    it[i] = item_of<VEC>(r, lane + (i << shift));
    if (lane + (i << shift) >= per) it[i] = Item{0, 0, 0, 0, false};
  }
}
// Both weights to LDS, each in its own weight_floats(dim) with zeros at their end.
__host__ __device__ inline int weight_floats(int dim) { return (dim + 3 & ~3) + 4; }
__device__ __forceinline__ void weights_to_lds(float *lds, const QkNormArgs &a) {
  const int each = weight_floats(a.r.dim);
#pragma unroll
  for (int kind = 0; kind < 2; ++kind)
    if (a.weight[kind])
      for (int i = threadIdx.x; i < each; i += 256) lds[kind * each + i] = i < a.r.dim ? a.weight[kind][i] : 0.0f;
}

// The coefficients of n tokens from t0 on, [n][half], and behind each token's zeros where a
// short vector's last channels would be.
constexpr int kCoefMore = 4;
template <typename IO, typename C2> __device__ __forceinline__ void form_coefficients(C2 *coef, const RotaryArgs &r, const FastDiv &half, int64_t t0, int n) {
  const int each = r.half + kCoefMore;
  for (int i = threadIdx.x; i < n * r.half; i += 256) {
    const int t = fast_div(i, half), j = i - t * r.half;
    C2 &to = coef[t * each + j];
    if constexpr (sizeof(C2) == sizeof(double2)) {
      double s, c;
      sincospi(2.0 * turn_fraction(r.positions[t0 + t], r.freqs[j]), &s, &c);
      to = make_double2((double)r.mscale * c, (double)r.mscale * s);
    } else if constexpr (sizeof(IO) == 4) {
      to = turn_fp32(r.positions[t0 + t], r.freqs[j], r.mscale, r.sign);
    } else {
      to = turn(r.positions[t0 + t], r.freqs[j], r.mscale, r.sign);
    }
  }
  for (int i = threadIdx.x; i < n * kCoefMore; i += 256) coef[i / kCoefMore * each + r.half + i % kCoefMore] = C2{0, 0};
}

// One workgroup: some tokens' rows, of queries, keys and, into pages, values.  The first
// rows are under way while the tokens' angles are formed, once for all heads, in LDS, and the
// next ones while a row is finished.
template <typename IO, int VEC, bool TAIL, int NI, int OUT>
__device__ __forceinline__ void forward_rows(const QkNormArgs &a, const QkNormPlan &p, int block, bool keys, float *weights, float2 *coef,
                                             int2 *place) {
  const RotaryArgs &r = a.r;
  const int64_t t0 = (int64_t)block * p.t.tokens[0];
  const int n = (int)(r.tokens - t0 < p.t.tokens[0] ? r.tokens - t0 : p.t.tokens[0]);
  const int shift = p.t.shift, lane = threadIdx.x & ((1 << shift) - 1), team = threadIdx.x >> shift, teams = 256 >> shift;
  const int nq = n * r.q_heads, nk = keys ? n * r.k_heads : 0, rows = nq + nk + (OUT == PAGES ? nk : 0);
  Item turned[NI], copied[NI];
  items_of<VEC>(p.t.per, p.t.shift, r, lane, turned);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    copied[i] = copy_of<VEC>(r, lane + (i << shift));
    if (copied[i].n0 <= 0) copied[i] = Item{0, 0, 0, 0, false};
  }
  struct Row {
    int kind, t, head;  // 0 a query, 1 a key, 2 a value
  };
  auto row_at = [&](int i) {
    Row w{0, 0, 0};
    if (i >= nq) {
      i -= nq;
      w.kind = 1;
      if (OUT == PAGES && i >= nk) {
        w.kind = 2;
        i -= nk;
      }
    }
    const int heads = w.kind ? r.k_heads : r.q_heads;
    w.t = fast_div(i, w.kind ? p.k_heads : p.q_heads);
    w.head = i - w.t * heads;
    return w;
  };
  auto items_for = [&](const Row &w, Item (&it)[NI]) {
    const bool copy = OUT == PAGES && w.kind == 2;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      it[i] = Item{copy ? copied[i].c0 : turned[i].c0, copy ? copied[i].c1 : turned[i].c1, copy ? copied[i].n0 : turned[i].n0,
                   copy ? copied[i].n1 : turned[i].n1, !copy && turned[i].turned};
  };
  using Raws = Raw<IO, VEC>[NI][2];
  auto load = [&](const Row &w, Raws &to) {
    const IO *src = (const IO *)(w.kind == 0 ? r.q : w.kind == 1 ? r.k : r.v) +
                    (t0 + w.t) * (w.kind == 0 ? r.q_stride : w.kind == 1 ? r.k_stride : r.v_stride) + (int64_t)w.head * r.dim;
    Item it[NI];
    items_for(w, it);
    load_row<IO, VEC, TAIL>(src, it, r.dim, to);
  };
  auto finish = [&](const Row &w, const Raws &from) {
    const int64_t tok = t0 + w.t;
    IO *dst;
    if (w.kind == 0) {
      dst = (IO *)r.q_out + (tok * r.q_heads + w.head) * r.dim;
    } else if (OUT == PACKED) {
      dst = (IO *)r.k_out + (tok * r.k_heads + w.head) * r.dim;
    } else {
      const int2 at = place[w.t];
      if (at.x < 0) return;
      dst = (IO *)(w.kind == 1 ? r.k_cache : r.v_cache) + (((int64_t)at.x * r.k_heads + w.head) * r.page + at.y) * r.dim;
    }
    Item it[NI];
    items_for(w, it);
    float x[NI][2][VEC];
    unpack_row<IO, VEC, TAIL>(from, it, r.dim, x);
    if (w.kind == 0 ? a.weight[0] != nullptr : w.kind == 1 && a.weight[1]) {
      const float rstd = rstd_of<float>(x, p.inv_dim, r.dim, a.eps, shift);
      weigh_row<float, VEC, TAIL>(x, rstd, weights + (w.kind ? weight_floats(r.dim) : 0), it, x);
    }
    const float2 *cf = coef + w.t * (r.half + kCoefMore);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (it[i].n0 > 0) {
        turn_item<VEC, TAIL>(it[i], r.interleaved, cf, x[i]);
        store_item<IO, VEC, TAIL>(dst, it[i], x[i]);
      }
  };
  Raws x0, x1;
  Row w0 = row_at(team < rows ? team : 0), w1;
  load(w0, x0);
  weights_to_lds(weights, a);
  form_coefficients<IO>(coef, r, p.half, t0, n);
  if (OUT != PACKED && (int)threadIdx.x < n) place[threadIdx.x] = place_of(r, t0 + threadIdx.x);
  __syncthreads();
  if (rows <= teams) {  // nothing to have under way
    if (team < rows) finish(w0, x0);
    return;
  }
  for (int row = team; row < rows; row += 2 * teams) {
    w1 = row_at(row + teams < rows ? row + teams : row);
    load(w1, x1);
    finish(w0, x0);
    if (row + teams >= rows) break;
    w0 = row_at(row + 2 * teams < rows ? row + 2 * teams : row);
    load(w0, x0);
    finish(w1, x1);
  }
}

// Keys into 4 bits: computed in 64 bits from their norm's sum to the rounding, so that a
// value next to the border of two codes, half a step apart, goes to the right one, which 32
// bits would miss once in some 10^5 values.  They pass through LDS, a wave's own part of it,
// where groups of 32 channels lie together whatever pairs were turned.  16384 tokens of 16
// query, 4 key and 4 value heads of 128: 50 us (3.7 TB/s), bound by instructions: the
// queries and values alone are 38, the keys and values 25, and waves of both share the SIMDs;
// in fp32, with twice the bytes a row, 72 us (5.0 TB/s).
// (fp32 first, its errors bounded, and 64 bits for the waves that have a value near a border,
// one in 50: 66 us, for most workgroups have such a wave and wait for it.)
__device__ __forceinline__ void wave_lds_ready() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
template <typename IO, int VEC, bool TAIL, int NI>
__device__ __forceinline__ void keys_to_fp4(const QkNormArgs &a, const QkNormPlan &p, int block, float *weights, double2 *coef,
                                            int2 *place, Upper *keys) {
  const RotaryArgs &r = a.r;
  const int64_t t0 = (int64_t)block * p.t.tokens[1];
  const int n = (int)(r.tokens - t0 < p.t.tokens[1] ? r.tokens - t0 : p.t.tokens[1]);
  const int shift = p.t.key_shift, lane = threadIdx.x & ((1 << shift) - 1), teams = 256 >> shift;
  const int in_wave = threadIdx.x & 63, wave_team = in_wave >> shift, wave_teams = 64 >> shift, rows = n * r.k_heads;
  Item it[NI];
  items_of<VEC>(p.t.key_per, shift, r, lane, it);
  Upper *const mine = keys + (threadIdx.x >> 6) * p.wave_keys;
  const int chunks = r.dim / 8, pieces = wave_teams * chunks;
  // A row lies as [8][chunks + 2], a channel's place in its piece first: lanes that read or
  // write one channel each of neighbouring pieces, or vectors, meet neighbouring banks.
  const int wave_row = 8 * (chunks + 2);
  auto place_in = [&](int c) { return (c & 7) * (chunks + 2) + (c >> 3); };
  using Raws = Raw<IO, VEC>[NI][2];
  auto load = [&](int row, Raws &to) {
    if (row >= rows) row = rows - 1;
    const int t = fast_div(row, p.k_heads), head = row - t * r.k_heads;
    load_row<IO, VEC, TAIL>((const IO *)r.k + (t0 + t) * r.k_stride + (int64_t)head * r.dim, it, r.dim, to);
  };
  // a wave's rows from row0 on
  auto finish = [&](int row0, const Raws &from) {
    const int row = row0 + wave_team;
    if (row < rows) {
      float x[NI][2][VEC];
      double y[NI][2][VEC];
      unpack_row<IO, VEC, TAIL>(from, it, r.dim, x);
      if (a.weight[1]) {
        const double rstd = rstd_of<double>(x, p.inv_dim, r.dim, a.eps, shift);
        weigh_row<double, VEC, TAIL>(x, rstd, weights + weight_floats(r.dim), it, y);
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[i][h][e] = x[i][h][e];
      }
      Upper *const to = mine + wave_team * wave_row;
      const double2 *const cf = coef + fast_div(row, p.k_heads) * (r.half + kCoefMore);
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (it[i].n0 > 0) {
          turn_item<VEC, TAIL>(it[i], r.interleaved, cf, y[i]);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            if (!TAIL || e < it[i].n0) to[place_in(it[i].c0 + e)] = upper(y[i][0][e]);
            if (e < it[i].n1) to[place_in(it[i].c1 + e)] = upper(y[i][1][e]);
          }
        }
    }
    wave_lds_ready();
    // four neighbouring lanes have a group; pieces are whole groups
    for (int i = in_wave; i < pieces; i += 64) {
      const int j = fast_div(i, p.chunks), chunk = i - j * chunks;
      if (row0 + j < rows) {
        const int t = fast_div(row0 + j, p.k_heads), head = row0 + j - t * r.k_heads;
        Upper x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = mine[j * wave_row + e * (chunks + 2) + chunk];
        store_fp4(a.k4, r, place[t], head, chunk, x);
      }
    }
    wave_lds_ready();
  };
  Raws x0, x1;
  int row0 = (threadIdx.x >> 6) * wave_teams;
  load(row0 + wave_team, x0);
  weights_to_lds(weights, a);
  form_coefficients<IO>(coef, r, p.half, t0, n);
  if ((int)threadIdx.x < n) place[threadIdx.x] = place_of(r, t0 + threadIdx.x);
  __syncthreads();
  for (; row0 < rows; row0 += 2 * teams) {
    load(row0 + teams + wave_team, x1);
    finish(row0, x0);
    if (row0 + teams >= rows) break;
    load(row0 + 2 * teams + wave_team, x0);
    finish(row0 + teams, x1);
  }
}

template <typename IO>
__device__ __forceinline__ void values_to_fp4(const QkNormArgs &a, const QkNormPlan &p, int block) {
  const RotaryArgs &r = a.r;
  const int token_items = r.k_heads * (r.dim / 8);
  const int64_t all = r.tokens * token_items;
  for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < all; i += (int64_t)p.t.blocks[2] * 256) {
    const int64_t tok = all <= INT32_MAX ? (int64_t)fast_div((uint32_t)i, p.v_items) : i / token_items;
    const int j = (int)(i - tok * token_items), head = fast_div(j, p.chunks), chunk = j - head * (r.dim / 8);
    const int2 at = place_of(r, tok);
    float x[8];
    Vec<IO, 8>::load((const IO *)r.v + tok * r.v_stride + (int64_t)head * r.dim + 8 * chunk, x);
    store_fp4(a.v4, r, at, head, chunk, x);
  }
}

template <typename IO, int VEC, bool TAIL, int NI, int OUT>
__global__ __launch_bounds__(256) void qk_norm_rotary_kernel(QkNormArgs a, QkNormPlan p) {
  extern __shared__ __align__(16) char lds[];  // weights, coefficients, places, keys on their way to codes
  float *const weights = reinterpret_cast<float *>(lds);
  char *const rest = lds + 2 * weight_floats(a.r.dim) * sizeof(float);
  float2 *const coef = reinterpret_cast<float2 *>(rest);
  if constexpr (OUT != PAGES4) {
    int2 *const place = reinterpret_cast<int2 *>(coef + p.t.tokens[0] * (a.r.half + kCoefMore));
    forward_rows<IO, VEC, TAIL, NI, OUT>(a, p, blockIdx.x, true, weights, coef, place);
  } else {
    int block = blockIdx.x;
    if (block < p.t.blocks[0]) {
      forward_rows<IO, VEC, TAIL, VEC == 8 ? 1 : NI, PACKED>(a, p, block, false, weights, coef, nullptr);
    } else if ((block -= p.t.blocks[0]) < p.t.blocks[1]) {
      double2 *const coef64 = reinterpret_cast<double2 *>(rest);
      int2 *const place = reinterpret_cast<int2 *>(coef64 + p.t.tokens[1] * (a.r.half + kCoefMore));
      keys_to_fp4<IO, 4, TAIL, NI>(a, p, block, weights, coef64, place, reinterpret_cast<Upper *>(place + p.t.tokens[1]));
    } else {
      values_to_fp4<IO>(a, p, block - p.t.blocks[1]);
    }
  }
}

// The reverse mode.  A workgroup passes its tokens a few at a time, the next ones' angles
// formed in the other half of LDS while rows are under way, and keeps both weights'
// gradients' sums of its rows in registers; it writes them once, as partial rows, which a
// second launch adds up in a fixed order.
template <typename IO, int VEC, bool TAIL, int NI>
__global__ __launch_bounds__(256) void qk_norm_rotary_bwd_kernel(QkNormArgs a, QkNormPlan p) {
  extern __shared__ __align__(16) char lds[];
  float *const weights = reinterpret_cast<float *>(lds);
  float2 *const coefs = reinterpret_cast<float2 *>(weights + 2 * weight_floats(a.r.dim));  // [2][tokens][half]
  __shared__ float cols[2][2][256 * VEC];
  const RotaryArgs &r = a.r;
  const int shift = p.t.shift, lane = threadIdx.x & ((1 << shift) - 1), team = threadIdx.x >> shift, teams = 256 >> shift;
  Item it[NI];
  items_of<VEC>(p.t.per, shift, r, lane, it);
  float dw[2][NI][2][VEC] = {};
  const int step = p.t.tokens[0], each = step * (r.half + kCoefMore);
  auto count = [&](int64_t t0) { return t0 >= r.tokens ? 0 : (int)(r.tokens - t0 < step ? r.tokens - t0 : step); };
  using Raws = Raw<IO, VEC>[NI][2];
  auto pass = [&](auto is_key, int64_t t0, int n, const float2 *coef, auto between) {
    constexpr int kKind = decltype(is_key)::value;
    const float *const weight = a.weight[kKind];
    const float *const wl = weights + kKind * weight_floats(r.dim);
    const int heads = kKind ? r.k_heads : r.q_heads, rows = n * heads;
    const IO *const xs = (const IO *)(kKind ? r.k : r.q) + t0 * (kKind ? r.k_stride : r.q_stride);
    const IO *const ds = (const IO *)a.dout[kKind] + t0 * a.dout_stride[kKind];
    IO *const to = (IO *)a.dx[kKind] + t0 * heads * r.dim;
    auto load = [&](int row, Raws &x, Raws &d) {
      const int t = fast_div(row, kKind ? p.k_heads : p.q_heads), head = row - t * heads;
      if (weight) load_row<IO, VEC, TAIL>(xs + t * (kKind ? r.k_stride : r.q_stride) + head * r.dim, it, r.dim, x);
      load_row<IO, VEC, TAIL>(ds + t * a.dout_stride[kKind] + head * r.dim, it, r.dim, d);
    };
    auto finish = [&](int row, const Raws &xr, const Raws &dr) {
      float x[NI][2][VEC], d[NI][2][VEC];
      unpack_row<IO, VEC, TAIL>(dr, it, r.dim, d);
      const float2 *const cf = coef + fast_div(row, kKind ? p.k_heads : p.q_heads) * (r.half + kCoefMore);
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (it[i].n0 > 0) turn_item<VEC, TAIL>(it[i], r.interleaved, cf, d[i]);
      if (weight) {
        unpack_row<IO, VEC, TAIL>(xr, it, r.dim, x);
        float wv[NI][2][VEC];
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            read_lds<VEC, !TAIL>(wl + (h ? it[i].c1 : it[i].c0), wv[i][h]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const float xe = x[i][h][e];
              ss = fused(xe, xe, ss);
              dot = fused(d[i][h][e] * wv[i][h][e], xe, dot);
            }
          }
        ss = team_sum(ss, shift);
        dot = team_sum(dot, shift);
        const float rstd = rsqrtf(fused(ss, p.inv_dim, a.eps));
        const float mean = dot * rstd * p.inv_dim;  // of dn n
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const float u = x[i][h][e] * rstd, de = d[i][h][e];
              dw[kKind][i][h][e] = fused(de, u, dw[kKind][i][h][e]);
              d[i][h][e] = rstd * fused(de, wv[i][h][e], -(u * mean));
            }
      }
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (it[i].n0 > 0) store_item<IO, VEC, TAIL>(to + row * r.dim, it[i], d[i]);
    };
    Raws x0, d0, x1, d1;
    if (rows > 0) load(team < rows ? team : 0, x0, d0);
    between();
    if (rows <= teams) {
      if (team < rows) finish(team, x0, d0);
      return;
    }
    for (int row = team; row < rows; row += 2 * teams) {
      load(row + teams < rows ? row + teams : row, x1, d1);
      finish(row, x0, d0);
      if (row + teams >= rows) break;
      load(row + 2 * teams < rows ? row + 2 * teams : row, x0, d0);
      finish(row + teams, x1, d1);
    }
  };
  int buf = 0;
  weights_to_lds(weights, a);
  form_coefficients<IO>(coefs, r, p.half, (int64_t)blockIdx.x * step, count((int64_t)blockIdx.x * step));
  __syncthreads();
  for (int64_t t0 = (int64_t)blockIdx.x * step; t0 < r.tokens; t0 += (int64_t)gridDim.x * step, buf ^= 1) {
    const float2 *const coef = coefs + buf * each;
    const int64_t next = t0 + (int64_t)gridDim.x * step;
    pass(std::integral_constant<int, 0>(), t0, count(t0), coef,
         [&] { form_coefficients<IO>(coefs + (buf ^ 1) * each, r, p.half, next, count(next)); });
    pass(std::integral_constant<int, 1>(), t0, count(t0), coef, [] {});
    __syncthreads();
  }
  // the teams' sums, an item of every thread at a time: of both kinds, both vectors.  Added in
  // 64 bits: 1531 tokens' keys' weights' gradients in fp32 are off by 1.2e-7 of themselves in
  // place of 1.6e-7, in the same time.
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (i > 0) __syncthreads();
#pragma unroll
    for (int kv = 0; kv < 4; ++kv)
#pragma unroll
      for (int e = 0; e < VEC; ++e) cols[kv / 2][kv % 2][threadIdx.x * VEC + e] = dw[kv / 2][i][kv % 2][e];
    __syncthreads();
    const int width = VEC << shift;
    for (int j = threadIdx.x; j < 4 * width; j += 256) {
      static_assert(VEC == 4);
      const int kv = j >> shift >> 2, kind = kv >> 1, h = kv & 1, at = j & (width - 1), item = at / VEC + (i << shift), e = at % VEC;
      if (!(kind ? a.weight[1] : a.weight[0]) || item >= p.t.per) continue;
      const Item part = item_of<VEC>(r, item);
      if (e >= (h ? part.n1 : part.n0)) continue;
      double s = 0.0;  // of up to 256 teams
      for (int k = 0; k < teams; ++k) s += cols[kind][h][(k << shift) * VEC + at];
      a.part[((int64_t)kind * gridDim.x + blockIdx.x) * r.dim + (h ? part.c1 : part.c0) + e] = (float)s;
    }
  }
}

// Rows of a cache in 4 bits as bf16 or fp32: 8 channels a thread.  16512 rows of 4 heads of
// 128, keys and values: 12.5 us, 3.8 TB/s, of which a launch's start and end are a third; 1152
// rows 3.3 us; in fp32 18.9 and 4.2 us.
template <typename IO>
__global__ __launch_bounds__(256) void cache_fp4_rows_kernel(Cache4Rows a, FastDiv chunks, FastDiv row_items) {
  const int per_row = a.heads * (a.dim / 8);
  const int side = blockIdx.y;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.rows * per_row; i += (int64_t)gridDim.x * 256) {
    const int64_t row = a.rows * per_row <= INT32_MAX ? (int64_t)fast_div((uint32_t)i, row_items) : i / per_row;
    const int j = (int)(i - row * per_row), head = fast_div(j, chunks), c = j - head * (a.dim / 8);
    const int64_t slot = a.slots[row];
    uint32_t v[4] = {0, 0, 0, 0};
    if (slot >= 0 && slot < a.num_pages * a.page) {
      const int64_t pg = a.num_pages * a.page <= INT32_MAX ? (int64_t)((uint32_t)slot / (uint32_t)a.page) : slot / a.page;
      const int64_t ph = pg * a.heads + head, at = slot - pg * a.page;
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

QkNormPlan plan_of(const QkNormArgs &a, const QkNormTiles &t) {
  const RotaryArgs &r = a.r;
  QkNormPlan p{};
  p.t = t;
  p.wave_keys = (64 >> t.key_shift) * (r.dim + 16);
  p.inv_dim = 1.0f / (float)r.dim;
  p.half = make_fast_div(r.half > 0 ? r.half : 1);
  p.q_heads = make_fast_div(r.q_heads);
  p.k_heads = make_fast_div(r.k_heads > 0 ? r.k_heads : 1);
  p.chunks = make_fast_div(r.dim >= 8 ? r.dim / 8 : 1);
  p.v_items = make_fast_div(r.k_heads > 0 && r.dim >= 8 ? r.k_heads * (r.dim / 8) : 1);
  return p;
}

// Whether `items` of each of a team's lanes are all of a head.
bool in_lanes(int items, int per, int shift) { return per <= items << shift; }

template <typename IO, int VEC, bool TAIL, int OUT> hipError_t forward(const QkNormArgs &a, const QkNormTiles &t, hipStream_t st) {
  const RotaryArgs &r = a.r;
  const QkNormPlan p = plan_of(a, t);
  const size_t weights = 2 * sizeof(float) * weight_floats(r.dim);
  size_t lds = weights + (size_t)t.tokens[0] * (sizeof(float2) * (r.half + kCoefMore) + sizeof(int2));
  if (OUT == PAGES4) {
    const size_t keys = weights + (size_t)t.tokens[1] * (sizeof(double2) * (r.half + kCoefMore) + sizeof(int2)) +
                        4 * p.wave_keys * sizeof(Upper);
    if (lds < keys) lds = keys;
  }
  const int grid = (int)(t.blocks[0] + t.blocks[1] + t.blocks[2]);
  // rows of vectors of 8 have one item a lane in every form; three are those of vectors of 4,
  // of the keys into 4 bits among them
  if (!in_lanes(VEC == 8 ? 1 : 3, t.per, t.shift) || !in_lanes(3, t.key_per, t.key_shift)) return hipErrorInvalidConfiguration;
  if (OUT == PAGES4 ? in_lanes(1, t.key_per, t.key_shift) : in_lanes(1, t.per, t.shift))
    qk_norm_rotary_kernel<IO, VEC, TAIL, 1, OUT><<<grid, 256, lds, st>>>(a, p);
  else if constexpr (VEC == 4 || OUT == PAGES4) qk_norm_rotary_kernel<IO, VEC, TAIL, 3, OUT><<<grid, 256, lds, st>>>(a, p);
  return hipGetLastError();
}
template <int OUT> hipError_t forward_form(const QkNormArgs &a, hipStream_t st) {
  const QkNormTiles t = qk_norm_tiles(a, false);
  if (!a.r.bf16) return t.tails ? forward<float, 4, true, OUT>(a, t, st) : forward<float, 4, false, OUT>(a, t, st);
  if (t.tails) return forward<u16, 4, true, OUT>(a, t, st);
  return t.vec == 8 ? forward<u16, 8, false, OUT>(a, t, st) : forward<u16, 4, false, OUT>(a, t, st);
}

template <typename IO, bool TAIL> hipError_t reverse(const QkNormArgs &a, const QkNormTiles &t, hipStream_t st) {
  const QkNormPlan p = plan_of(a, t);
  const size_t lds = 2 * sizeof(float) * weight_floats(a.r.dim) + 2 * sizeof(float2) * (size_t)t.tokens[0] * (a.r.half + kCoefMore);
  if (!in_lanes(3, t.per, t.shift)) return hipErrorInvalidConfiguration;
  if (in_lanes(1, t.per, t.shift)) qk_norm_rotary_bwd_kernel<IO, 4, TAIL, 1><<<(int)t.blocks[0], 256, lds, st>>>(a, p);
  else qk_norm_rotary_bwd_kernel<IO, 4, TAIL, 3><<<(int)t.blocks[0], 256, lds, st>>>(a, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm_rotary(const QkNormArgs &a, hipStream_t st) {
  if (a.r.tokens == 0) return hipSuccess;
  TimedLaunch tl(K_QK_NORM, st);
  if (a.into4) return forward_form<PAGES4>(a, st);
  return a.r.slots ? forward_form<PAGES>(a, st) : forward_form<PACKED>(a, st);
}

hipError_t launch_qk_norm_rotary_bwd(const QkNormArgs &a, hipStream_t st) {
  TimedLaunch tl(K_QK_NORM_BWD, st);
  const QkNormTiles t = qk_norm_tiles(a, true);
  if (a.r.tokens > 0) {
    const hipError_t e = a.r.bf16 ? (t.tails ? reverse<u16, true>(a, t, st) : reverse<u16, false>(a, t, st))
                                  : t.tails ? reverse<float, true>(a, t, st) : reverse<float, false>(a, t, st);
    if (e != hipSuccess) return e;
  }
  if (!a.weight[0] && !a.weight[1]) return hipSuccess;
  return launch_norm_partials(a.part, (int)t.blocks[0], a.r.dim,
                              {a.weight[0] ? a.dweight[0] : nullptr, a.weight[1] ? a.dweight[1] : nullptr, nullptr}, st);
}

hipError_t launch_cache_fp4_rows(const Cache4Rows &a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  TimedLaunch tl(K_CACHE_FP4_ROWS, st);
  const int64_t items = a.rows * a.heads * (a.dim / 8), blocks = (items + 255) / 256;
  const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384), a.out[1] ? 2 : 1);
  const FastDiv chunks = make_fast_div(a.dim / 8), row_items = make_fast_div(a.heads * (a.dim / 8));
  if (a.bf16) cache_fp4_rows_kernel<u16><<<grid, 256, 0, st>>>(a, chunks, row_items);
  else cache_fp4_rows_kernel<float><<<grid, 256, 0, st>>>(a, chunks, row_items);
  return hipGetLastError();
}

}  // namespace flare
