// host_layer.cpp -- validation of the operators around the GDN step before any
// launch, how they are cut into work, and the workspace sizes that follow.
// Pure C++.
#include "block_attn.h"
#include "host_plan.h"

namespace flare {

namespace {
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
}  // namespace

AttnPlan attn_plan(const BlockAttnArgs &a) {
  AttnPlan p{};
  while ((1 << p.page_shift) < a.page) ++p.page_shift;
  const int64_t rows = (int64_t)a.block * (a.q_heads / a.kv_heads);
  const int64_t all_rows = rows * a.num_req;
  // Two row tiles a wave where that leaves a workgroup for every CU: half the reads of
  // K and V.  30 requests x 32, 32 query and 4 kv heads of 128, 1000 own keys (240
  // workgroups of two): 26 us with one, 39 with two; 60 requests (480): 50 and 44.
  p.own_tiles = a.dim <= 128 && rows > 64 && ceil_div(rows, 128) * a.kv_heads * a.num_req >= 256 ? 2 : 1;
  p.prefix_tiles = a.dim <= 128 && (all_rows > 64 || p.own_tiles == 2) ? 2 : 1;
  p.own_groups = (int)ceil_div(rows, 64 * p.own_tiles);
  p.prefix_groups = (int)ceil_div(all_rows, 64 * p.prefix_tiles);
  // a wave keeps the pages of its part's tiles in its 64 lanes
  const int64_t longest = a.dim == 256 ? 2048 : 4096;

  // How long the parts are: the shortest time, counted in keys that a workgroup
  // passes (64 in about 1.3 us).  512 workgroups run at a time (two a CU); one costs
  // its keys and 384 more for its start and end; the whole takes no less than all of
  // them over the 512, nor than the rounds of either kind alone; and every part is
  // written and read again by the joining launch, rows * dim * 8 bytes at 5 TB/s and a
  // little.  Measured, with the chosen lengths first:
  //   256 requests x 4 (16 q, 4 kv heads, d = 128), prefix 8192, own 1024: prefix parts
  //   of 4096 120 us, 2048 131, 1024 152 (long ones leave a slot of every CU to the
  //   own keys throughout); 16 x 4 over 4096 own keys: parts of 512 27.0 us, 256 31.1,
  //   1024 29.8; 16 x 4 over a prefix of 4096: 256 21.5 us, 128 24.6, 512 24.4;
  //   37 x 7 at d = 256, own 777: parts of 512 41 us, 128 50.
  constexpr int64_t kSlots = 512, kStart = 384;
  const int64_t join = all_rows * a.kv_heads * a.dim / 12500 + 2;
  const int64_t units = (int64_t)p.own_groups * a.kv_heads * a.num_req;
  p.prefix_chunk = p.own_chunk = (int)longest;
  int64_t best = INT64_MAX, own_top = longest;
  while (own_top > 128 && own_top / 2 >= a.max_seq_len) own_top /= 2;
  const int64_t least = ceil_div(a.prefix_len, longest), most = ceil_div(a.prefix_len, 128);
  for (int64_t n = least; n <= most; n += 1 + n / 4) {
    // a unit (kv head, part) of the prefix stays on one of 8 XCDs
    const int64_t chunk = n > 0 ? ceil_div(ceil_div(a.prefix_len, n), 64) * 64 : longest;
    const int64_t parts = ceil_div(a.prefix_len, chunk), units8 = ceil_div(parts * a.kv_heads, 8) * p.prefix_groups;
    const int64_t prefix_rounds = ceil_div(units8, kSlots / 8) * (chunk + kStart);
    for (int64_t c = own_top; c >= 128; c /= 2) {
      const int64_t own_parts = ceil_div(a.max_seq_len, c);
      const int64_t own_keys = (c < a.max_seq_len ? c : a.max_seq_len) + kStart;
      int64_t cost = (8 * units8 * (chunk + kStart) + units * own_parts * own_keys) / kSlots;
      const int64_t own_rounds = ceil_div(units * own_parts, kSlots) * own_keys;
      if (parts > 0 && cost < prefix_rounds) cost = prefix_rounds;
      if (cost < own_rounds) cost = own_rounds;
      cost += (parts + own_parts) * join;
      if (cost < best) {
        best = cost;
        p.prefix_chunk = (int)chunk;
        p.prefix_parts = (int)parts;
        p.own_chunk = (int)c;
        p.own_parts = (int)own_parts;
      }
    }
  }
  p.prefix_blocks = ceil_div((int64_t)p.prefix_parts * a.kv_heads, 8) * 8 * p.prefix_groups;
  // A short prefix is passed by every request before its own keys, in one part: no
  // join and no second launch, where that takes less than its sharing does.
  const int64_t tile = a.dim == 256 ? 32 : 64;
  if (a.prefix_len > 0 && ceil_div(a.prefix_len, tile) + ceil_div(a.max_seq_len, tile) <= 64) {
    const int64_t together = ceil_div(units, kSlots) * (a.prefix_len + a.max_seq_len + kStart);
    const int64_t apart = best + kStart;  // and the second launch
    if (together <= apart) {
      p.merged = 1;
      p.prefix_parts = 0;
      p.prefix_blocks = 0;
      p.own_parts = 1;
      p.own_chunk = (int)longest;
    }
  }
  if (p.prefix_parts + p.own_parts == 0) p.own_parts = 1;  // no keys at all: zeros are written
  p.own_blocks = units * p.own_parts;
  p.prefix_runs = (int)ceil_div(p.prefix_blocks, 8 * kOctets);
  p.own_runs = (int)ceil_div(p.own_blocks, 8 * kOctets);
  return p;
}

int64_t attn_launch_blocks(const AttnPlan &p) {
  const int64_t run = 8 * kOctets;
  return (ceil_div(p.prefix_blocks, run) + ceil_div(p.own_blocks, run)) * run;
}

int norm_bwd_blocks(int64_t rows, int32_t dim) {
  // what the chip holds at a time: six workgroups of 256 threads a CU where a wave or
  // two hold a row, three where a row is the workgroup's
  const int64_t most = dim <= 1024 ? 1536 : 768;
  return (int)(rows < most ? rows : most);
}

size_t norm_bwd_workspace_bytes(int64_t rows, int32_t dim, int weights) {
  return (size_t)norm_bwd_blocks(rows, dim) * dim * weights * sizeof(float) + 256;
}

flare_status check_io(int32_t io_dtype) {
  if (io_dtype != FLARE_F32 && io_dtype != FLARE_BF16)
    return fail(FLARE_ERR_UNSUPPORTED, "io_dtype %d unknown", io_dtype);
  return FLARE_OK;
}

flare_status check_gate(const void *gate, int32_t activation, int64_t stride, int64_t row) {
  if (!gate) return FLARE_OK;
  if (activation != FLARE_GATE_LINEAR && activation != FLARE_GATE_SILU && activation != FLARE_GATE_SIGMOID)
    return fail(FLARE_ERR_UNSUPPORTED, "gate activation %d unknown", activation);
  if (stride < row) return fail(FLARE_ERR_SHAPE, "gate_stride %lld below a row of %lld", (long long)stride, (long long)row);
  return FLARE_OK;
}

flare_status check_eps(float eps) {
  if (!(eps >= 0.0f && eps < 1e30f)) return fail(FLARE_ERR_SHAPE, "eps must be a number of at least 0");
  return FLARE_OK;
}

static flare_status check_norm_rows(int64_t rows, int32_t dim, int64_t x_stride, int64_t row) {
  if (dim < 1) return fail(FLARE_ERR_SHAPE, "dim must be positive");
  if (dim > 16384) return fail(FLARE_ERR_UNSUPPORTED, "dim %d, at most 16384", dim);
  if (rows > INT32_MAX) return fail(FLARE_ERR_UNSUPPORTED, "%lld rows, at most 2^31 - 1", (long long)rows);
  if (x_stride < row) return fail(FLARE_ERR_SHAPE, "x_stride %lld below a row of %lld", (long long)x_stride, (long long)row);
  return FLARE_OK;
}

flare_status check_gated_norm(int64_t tokens, int32_t heads, int32_t dim, int32_t io_dtype, const void *x,
                              int64_t x_stride, const void *gate, int64_t gate_stride, const float *weight,
                              int32_t activation) {
  if (tokens < 0 || heads < 1) return fail(FLARE_ERR_SHAPE, "tokens must not be negative, heads positive");
  if (tokens > INT32_MAX) return fail(FLARE_ERR_UNSUPPORTED, "too many tokens");
  const int64_t row = (int64_t)heads * (dim > 0 ? dim : 0);
  flare_status st = check_io(io_dtype);
  if (st != FLARE_OK) return st;
  st = check_norm_rows(tokens * heads, dim, x_stride, row);
  if (st != FLARE_OK) return st;
  st = check_gate(gate, activation, gate_stride, row);
  if (st != FLARE_OK) return st;
  if (tokens > 0 && (!x || !weight)) return fail(FLARE_ERR_NULL, "gated_norm: a required pointer is NULL");
  return FLARE_OK;
}

flare_status check_residual_norm(int64_t tokens, int32_t dim, int32_t io_dtype, int32_t res_dtype, const void *x,
                                 int64_t x_stride, const void *residual, const void *gate, int64_t gate_stride,
                                 const float *w_pre, int32_t activation) {
  if (tokens < 0) return fail(FLARE_ERR_SHAPE, "tokens must not be negative");
  flare_status st = check_io(io_dtype);
  if (st == FLARE_OK) st = check_io(res_dtype);
  if (st != FLARE_OK) return st;
  if (res_dtype == FLARE_BF16 && io_dtype != FLARE_BF16)
    return fail(FLARE_ERR_UNSUPPORTED, "a bf16 residual goes with bf16 io");
  st = check_norm_rows(tokens, dim, x_stride, dim);
  if (st != FLARE_OK) return st;
  st = check_gate(gate, activation, gate_stride, dim);
  if (st != FLARE_OK) return st;
  if (tokens > 0 && (!x || !residual || !w_pre))
    return fail(FLARE_ERR_NULL, "residual_norm: a required pointer is NULL");
  return FLARE_OK;
}

flare_status check_workspace(const void *workspace, size_t bytes, size_t need) {
  if (!workspace || bytes < need)
    return fail(FLARE_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? bytes : (size_t)0, need);
  if (((uintptr_t)workspace & 255u) != 0) return fail(FLARE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  return FLARE_OK;
}

flare_status check_rotary(int64_t tokens, const flare_rotary_shape *s, const int32_t *positions, const double *freqs,
                          const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *q_out) {
  if (!s) return fail(FLARE_ERR_NULL, "rotary: shape is NULL");
  if (tokens < 0 || s->q_heads < 1 || s->k_heads < 0 || s->dim < 1 || s->half < 0)
    return fail(FLARE_ERR_SHAPE, "rotary: negative sizes, or no q heads or channels");
  if (tokens > INT32_MAX) return fail(FLARE_ERR_UNSUPPORTED, "rotary: too many tokens");
  if (s->dim > 1024) return fail(FLARE_ERR_UNSUPPORTED, "rotary: dim %d, at most 1024", s->dim);
  if (s->q_heads > 65536 || s->k_heads > 65536) return fail(FLARE_ERR_UNSUPPORTED, "rotary: at most 65536 heads");
  if (s->half > s->dim / 2)  // 2 * half itself can pass 32 bits
    return fail(FLARE_ERR_SHAPE, "rotary: half = %d, of a head of %d channels", s->half, s->dim);
  if (s->interleaved != 0 && s->interleaved != 1)
    return fail(FLARE_ERR_UNSUPPORTED, "rotary: interleaved %d unknown", s->interleaved);
  flare_status st = check_io(s->io_dtype);
  if (st != FLARE_OK) return st;
  if (q_stride < (int64_t)s->q_heads * s->dim || (s->k_heads > 0 && k_stride < (int64_t)s->k_heads * s->dim))
    return fail(FLARE_ERR_SHAPE, "rotary: a token stride is below a row");
  if (tokens > 0 && (!positions || (s->half > 0 && !freqs) || !q || !q_out || (s->k_heads > 0 && !k)))
    return fail(FLARE_ERR_NULL, "rotary: a required pointer is NULL");
  return FLARE_OK;
}

int rotary_block_tokens(const RotaryArgs &a) {
  // more tokens a workgroup while its work items stay below two a thread and 1024
  // workgroups are left: 65536 tokens of 6 heads of 64, 1 to 16 of them: 55, 32, 25, 22,
  // 20 us; 32768 of 20 heads of 128: 71, 62, 63, 65, 74
  const int items = rotary_items(a, rotary_vec(a.bf16)).token;
  int tb = 1;
  while (tb < 16 && 2 * tb * items <= 512 && a.tokens / (2 * tb) >= 1024 && 2 * tb * a.half <= 2048) tb *= 2;
  return tb;
}

flare_status check_rotary_blocks(const RotaryArgs &a) {
  const int64_t tb = rotary_block_tokens(a);
  if (ceil_div(a.tokens, tb) > kMaxBlocks)
    return fail(FLARE_ERR_UNSUPPORTED, "rotary: %lld tokens, at most %lld of so many heads", (long long)a.tokens,
                (long long)(kMaxBlocks * tb));
  return FLARE_OK;
}

flare_status check_step_tables(const StepTablesArgs &a) {
  if (a.num_req < 0 || a.max_pages < 0 || a.num_free < 0 || a.max_tokens < 0 || a.position_offset < 0)
    return fail(FLARE_ERR_SHAPE, "step_tables: a negative size");
  if (a.page < 1) return fail(FLARE_ERR_SHAPE, "step_tables: page must be positive");
  if (a.num_req > kTablesMaxReq)
    return fail(FLARE_ERR_UNSUPPORTED, "step_tables: %d requests, at most %d", a.num_req, kTablesMaxReq);
  if (a.num_free > INT32_MAX || a.max_tokens > INT32_MAX)
    return fail(FLARE_ERR_UNSUPPORTED, "step_tables: at most 2^31 - 1 free pages and tokens");
  if (!a.pages_used || !a.pages_used_out || !a.status || !a.cu_new ||
      (a.num_req > 0 && (!a.seq_lens || !a.new_lens || !a.seq_lens_out)) || (a.num_req > 0 && a.max_pages > 0 && !a.block_table) ||
      (a.num_free > 0 && !a.free_pages) || (a.max_tokens > 0 && (!a.positions || !a.slots)))
    return fail(FLARE_ERR_NULL, "step_tables: a required pointer is NULL");
  if (a.pages_used == a.pages_used_out ||
      (a.num_req > 0 && (a.seq_lens == a.seq_lens_out || a.new_lens == a.seq_lens_out)))
    return fail(FLARE_ERR_SHAPE, "step_tables: an output is the memory of its input");
  return FLARE_OK;
}

flare_status check_attention_shape(int32_t num_req, const flare_attention_shape *s, int32_t max_seq_len,
                                   int32_t prefix_len) {
  if (!s) return fail(FLARE_ERR_NULL, "block_attention: shape is NULL");
  if (num_req < 0 || max_seq_len < 0 || prefix_len < 0) return fail(FLARE_ERR_SHAPE, "block_attention: a negative size");
  if (s->block < 1 || s->q_heads < 1 || s->kv_heads < 1)
    return fail(FLARE_ERR_SHAPE, "block_attention: block and heads must be positive");
  if (s->q_heads % s->kv_heads != 0)
    return fail(FLARE_ERR_SHAPE, "block_attention: %d q heads are no multiple of %d kv heads", s->q_heads, s->kv_heads);
  if (s->head_dim != 64 && s->head_dim != 128 && s->head_dim != 256)
    return fail(FLARE_ERR_UNSUPPORTED, "block_attention: head dim %d not instantiated (64, 128, 256)", s->head_dim);
  if (s->page < 16 || (s->page & (s->page - 1)) != 0)
    return fail(FLARE_ERR_UNSUPPORTED, "block_attention: page %d is no power of two of at least 16", s->page);
  if (s->io_dtype != FLARE_BF16) return fail(FLARE_ERR_UNSUPPORTED, "block_attention: bf16 only");
  if (!(s->scale < 1e30f) || s->scale < -1e30f)
    return fail(FLARE_ERR_SHAPE, "block_attention: scale must be a number below 1e30");
  if (s->causal != 0 && s->causal != 1) return fail(FLARE_ERR_UNSUPPORTED, "block_attention: causal %d unknown", s->causal);
  // keys are counted in 32 bits, with room for a tile past the end
  if (max_seq_len > INT32_MAX - 8192 || prefix_len > INT32_MAX - 8192)
    return fail(FLARE_ERR_UNSUPPORTED, "block_attention: at most 2^31 - 8193 keys");
  if ((int64_t)num_req * s->block > INT32_MAX / 64 / s->q_heads)
    return fail(FLARE_ERR_UNSUPPORTED, "block_attention: num_req * block * q_heads beyond 2^25");
  return FLARE_OK;
}

BlockAttnArgs attention_args(int32_t num_req, const flare_attention_shape *s, int32_t max_seq_len,
                             int32_t prefix_len) {
  BlockAttnArgs a{};
  a.num_req = num_req;
  a.block = s->block;
  a.q_heads = s->q_heads;
  a.kv_heads = s->kv_heads;
  a.dim = s->head_dim;
  a.page = s->page;
  a.causal = s->causal;
  a.prefix_len = prefix_len;
  a.max_seq_len = max_seq_len;
  a.scale = s->scale > 0.0f ? s->scale : 1.0f / __builtin_sqrtf((float)s->head_dim);
  return a;
}

size_t block_attention_workspace_bytes(const BlockAttnArgs &a, const AttnPlan &p) {
  const int64_t parts = (int64_t)p.prefix_parts + p.own_parts;
  if (a.num_req == 0 || parts <= 1) return 0;
  return (size_t)parts * a.num_req * a.block * a.q_heads * (a.dim + 2) * sizeof(float) + 256;
}

}  // namespace flare
