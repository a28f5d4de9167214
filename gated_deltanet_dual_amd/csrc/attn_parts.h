// attn_parts.h -- what the block attentions share: how a launch's workgroups find their
// part, and the exchanges of a softmax whose lanes keep a query each.
#pragma once

#include "block_attn.h"
#include "device_common.h"

namespace flare {

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

// Two weights of at least 0 in two bf16 halves each, the first ones in x: cut, so that up to
// 2^-7 of a weight is left, and that rounded, off by 2^-15 of the weight at most.  2^-20 of it
// are added, so that the second half of a weight above 2^-113 is above 0 as well: a value of
// infinity times both halves stays one.
__device__ __forceinline__ uint2 two_halves(float x, float y) {
  const uint32_t first = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
  constexpr float kMore = 1.0f + 0x1p-20f;
  return make_uint2(first, pack_bf16x2(__builtin_fmaf(x, kMore, -__uint_as_float(first << 16)),
                                       __builtin_fmaf(y, kMore, -__uint_as_float(first & 0xffff0000u))));
}

// What a workgroup works on: rows [row0, row_end) (token * G + query of the
// group) of one kv head against keys [k0, k1) of the prefix or of one request.
struct Part {
  uint32_t row0, row_end;
  int head, k0, k1, out;  // out: the part's place in the workspace
  int pre;                // keys of the prefix that come before k0 (a short prefix, not shared)
  int len, req;           // own keys of the request; req < 0: the prefix
  const int32_t *table;
};

// The id-th workgroup of the requests' own keys.
template <int OWN_ROWS>
__device__ __forceinline__ bool own_part(const BlockAttnArgs &a, const AttnPlan &p, uint32_t id, Part &w) {
  const uint32_t BG = a.block * (a.q_heads / a.kv_heads);
  if (id >= p.own_blocks) return false;
  w.head = (int)(id % (uint32_t)a.kv_heads);
  id /= (uint32_t)a.kv_heads;
  const uint32_t rg = id % (uint32_t)p.own_groups;
  id /= (uint32_t)p.own_groups;
  // all requests' first parts before their second: the longest requests' last ones start last
  w.req = (int)(id % (uint32_t)a.num_req);
  const int part = (int)(id / (uint32_t)a.num_req);
  w.len = attn_own_len(a, a.seq_lens[w.req]);
  w.row0 = w.req * BG + rg * OWN_ROWS;
  w.row_end = (w.req + 1) * BG;
  w.k0 = part * p.own_chunk;
  w.k1 = w.len - w.k0 < p.own_chunk ? w.len : w.k0 + p.own_chunk;
  w.out = p.prefix_parts + part;
  w.pre = p.merged ? a.prefix_len : 0;
  w.table = a.block_table + (int64_t)w.req * a.max_pages;
  // a part behind the request's length is not read by the joining launch; the
  // only part is written in any case
  return w.k0 < w.k1 || p.prefix_parts + p.own_parts == 1;
}

// Workgroups of the prefix and of the requests' own keys alternate in runs of one
// workgroup for each CU, in proportion and the prefix first: the prefix is bound by
// its products, the own keys by memory, so a CU holds both kinds at a time (256
// requests x 4, 16 query and 4 kv heads of 128, prefix 8192 and own 1024: 120 us
// where alternating octets, which leave some CUs two of a kind, took 145).  The units
// (head, part) of the prefix go round the XCDs and a unit's row groups stay on one:
// they read the same keys from its L2.
template <int PREFIX_ROWS, int OWN_ROWS>
__device__ __forceinline__ bool find_part(const BlockAttnArgs &a, const AttnPlan &p, Part &w) {
  const uint32_t G = a.q_heads / a.kv_heads, BG = a.block * G;
  const uint32_t run = blockIdx.x / 8 / kOctets, in = blockIdx.x / 8 % kOctets, all = p.prefix_runs + p.own_runs;
  const uint32_t before = ((uint64_t)run * p.prefix_runs + all - 1) / all;  // runs of the prefix before this one
  if (((uint64_t)(run + 1) * p.prefix_runs + all - 1) / all > before) {
    const uint32_t pi = before * kOctets + in;
    const uint32_t unit = pi / p.prefix_groups * 8 + blockIdx.x % 8, rg = pi % p.prefix_groups;
    if (unit >= (uint32_t)(a.kv_heads * p.prefix_parts)) return false;
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
  return own_part<OWN_ROWS>(a, p, ((run - before) * kOctets + in) * 8 + blockIdx.x % 8, w);
}

}  // namespace flare
