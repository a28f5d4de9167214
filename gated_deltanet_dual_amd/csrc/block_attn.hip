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

#include "attn_tiles.h"
#include "device_common.h"
#include "layer_launch.h"

namespace flare {
namespace {

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
// The tiles of a bf16 cache, which memory fills straight into LDS.  TK = 64: a wave fills
// one subtile of K and of V; TK = 32: waves 0, 1 fill K, 2, 3 V.  A lane fetches the piece of
// its row that k_piece / v_piece put where it lands.  Row and piece of load i differ from
// those of load 0 by bits of i alone, so the byte offset is that of load 0 with a constant's
// bits turned over.
template <int D, int TK, bool NT> struct MemoryToLds {
  static constexpr int SUBS = TK / 16, PIECES = D / 8, RPI = 64 / PIECES;
  static constexpr int LOADS = 16 * PIECES / 64;  // 1 KiB loads of a subtile
  const BlockAttnArgs &a;
  int shift, wave;
  uint32_t ky, vy, k_at, v_at;
  __device__ __forceinline__ MemoryToLds(const BlockAttnArgs &a, int shift, int lane, int wave, int sub, const u16 (&kt_lds)[2][TK * D],
                                         const u16 (&vt_lds)[2][TK * D])
      : a(a), shift(shift), wave(wave) {
    ky = 2 * (lane / PIECES * D + k_piece<D>(lane / PIECES, lane % PIECES) * 8);
    vy = 2 * (lane / PIECES * D + v_piece<D>(lane / PIECES, lane % PIECES) * 8);
    k_at = lds_at(&kt_lds[0][sub * 16 * D]);
    v_at = lds_at(&vt_lds[0][sub * 16 * D]);
  }
  __device__ __forceinline__ void load(int pg, int head, int row, int buf) const {
    const int64_t at = ((((int64_t)pg * a.kv_heads + head) << shift) + row) * D;
    const u16 *kp = uniform((const u16 *)a.k_cache + at), *vp = uniform((const u16 *)a.v_cache + at);
    const uint32_t to = buf * (TK * D * 2);
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
  }
  static constexpr bool kLands = false, kHalves = false;
};

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
  if (w.req < 0 || (NQP == NQO && !NT)) attn_part<D, NQP, TK, MemoryToLds<D, TK, false>>(a, p, w, turn, kt_lds, vt_lds);
  else attn_part<D, NQO, TK, MemoryToLds<D, TK, NT>>(a, p, w, turn, kt_lds, vt_lds);
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
