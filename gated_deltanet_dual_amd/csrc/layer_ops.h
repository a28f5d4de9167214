// layer_ops.h -- argument blocks and launchers of the operators around the GDN
// step (norms, rotary positions, serving-step tables, block attention), and
// their host-side checks.  Internal.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/flare_gdn.h"

#ifdef __HIPCC__
#define FLARE_HD __host__ __device__ inline
#else
#define FLARE_HD inline
#endif

namespace flare {

// ---------------------------------------------------------------- norms

struct GatedNormArgs {
  int64_t tokens;
  int heads, dim, bf16, act;  // act: -1 without a gate, else FLARE_GATE_*
  float eps;
  const void *x, *gate, *dy;
  int64_t x_stride, gate_stride, dy_stride;  // elements between tokens
  const float *weight;
  float *rstd;  // forward: written (or NULL); reverse: read
  void *y, *dx, *dgate;
  float *dweight, *part;  // part [blocks][dim]
};

struct ResidualNormArgs {
  int64_t tokens;
  int dim, bf16, res_bf16, act;  // act: -1 without a gate
  float eps;
  const void *x, *residual, *gate, *dy, *dh;  // dh NULL = 0
  int64_t x_stride, gate_stride;
  const float *w_pre, *w_post, *scale;  // w_post, scale NULL = absent
  float *rstd;                          // [tokens][2]: post, pre
  void *h, *y, *dx, *dres, *dgate;
  float *dw_pre, *dw_post, *dscale;
  float *part[3];  // [blocks][dim] of w_pre, w_post, scale; the workspace in part[0] at the launcher
};

// ---------------------------------------------------------------- rotary
struct RotaryArgs {
  int64_t tokens;
  int q_heads, k_heads, dim, half, bf16, interleaved;
  float mscale, sign;
  const int32_t *positions;
  const double *freqs;  // [half] radians per position
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  void *q_out, *k_out;
  // into the cache instead of k_out: row t to slot slots[t]; slots outside
  // [0, num_pages * page) write nothing
  const int64_t *slots;
  void *k_cache, *v_cache;
  int64_t num_pages;
  int page;
};

// A head's work items hold two vectors each, so that a thread has two loads in
// flight.  First those that turn: a vector of each half, or in the interleaved
// layout two whole vectors; then copies.  The last vectors can be short.
FLARE_HD int rotary_vectors(int channels, int vec) { return (channels + vec - 1) / vec; }
FLARE_HD int rotary_turned_items(const RotaryArgs &a, int vec) {
  return a.interleaved ? (rotary_vectors(2 * a.half, vec) + 1) / 2 : rotary_vectors(a.half, vec);
}
FLARE_HD int rotary_copy_items(int channels, int vec) { return (rotary_vectors(channels, vec) + 1) / 2; }

struct RotaryItems {
  int per, v_per, token;  // work items of a q or k head, of a v head (0: none) and of a token
};
FLARE_HD RotaryItems rotary_items(const RotaryArgs &a, int vec) {
  const int per = rotary_turned_items(a, vec) + rotary_copy_items(a.dim - 2 * a.half, vec);
  const int v_per = a.slots ? rotary_copy_items(a.dim, vec) : 0;
  return {per, v_per, (a.q_heads + a.k_heads) * per + a.k_heads * v_per};
}
constexpr int rotary_vec(bool bf16) { return bf16 ? 8 : 4; }  // 16 bytes
int rotary_block_tokens(const RotaryArgs &a);                 // tokens a workgroup

// ---------------------------------------------------------------- q/k norms with rotary positions
// A cache in 4 bits: rows of dim / 2 bytes of codes, and for each group of 32
// channels a page's bytes of scales.
struct Cache4 {
  uint8_t *codes;   // [num_pages, heads, page, dim / 2]
  uint8_t *scales;  // [num_pages, heads, dim / 32, page]
};

struct QkNormArgs {
  RotaryArgs r;  // sizes, positions, q, k, v, where they go; the reverse mode's sign is -1
  float eps;
  const float *weight[2];  // of q and k; NULL: turned, not normed
  bool into4;              // k4, v4 in place of r.k_cache, r.v_cache
  Cache4 k4, v4;
  // reverse mode: the gradients of the outputs, then of the inputs
  const void *dout[2];
  int64_t dout_stride[2];
  void *dx[2];
  float *dweight[2], *part;  // part [2][blocks][dim]
};

// How the work is dealt.  A row goes to a team of 1 << shift lanes, its items of two vectors
// one a lane, and a workgroup has some tokens' rows at a time.
struct QkNormTiles {
  int vec;     // channels of a vector
  bool tails;  // short vectors occur
  int per;     // work items of a head
  int shift;
  int key_per, key_shift;  // of keys into 4 bits, whose vectors have 4 channels
  int tokens[2];      // of a workgroup; into 4 bits those of queries and of keys
  int64_t blocks[3];  // workgroups; into 4 bits those of queries, keys and values follow each other
};
QkNormTiles qk_norm_tiles(const QkNormArgs &a, bool reverse);

struct Cache4Rows {
  int64_t rows, num_pages;
  int heads, dim, page, bf16;
  const int64_t *slots;
  const uint8_t *codes[2], *scales[2];  // of keys and values; out[1] NULL: keys alone
  void *out[2];                         // [rows, heads, dim]
};

// ---------------------------------------------------------------- step tables
constexpr int kTablesMaxReq = 8192;  // three int32 per request in LDS

struct StepTablesArgs {
  int num_req, max_pages, page;
  int64_t num_free, max_tokens;
  int position_offset;
  const int32_t *seq_lens, *new_lens, *free_pages, *pages_used;
  int32_t *block_table, *cu_new, *positions, *seq_lens_out, *pages_used_out, *status;
  int64_t *slots;
};

// ---------------------------------------------------------------- attention
struct BlockAttnArgs {
  int num_req, block, q_heads, kv_heads, dim, page, max_pages, causal;
  int64_t num_pages;
  int prefix_len, max_seq_len;
  float scale;
  const void *q, *k_cache, *v_cache;
  const int32_t *block_table, *seq_lens, *prefix_table;
  void *o;
  float *lse;
  float *part;  // workspace
};

struct BlockAttnFp4Args {
  BlockAttnArgs a;  // its caches are the codes
  const uint8_t *k_scales, *v_scales;
};

// ---------------------------------------------------------------- host checks
// A launch dimension holds fewer than 2^32 work items: so many workgroups of 256.
constexpr int64_t kMaxBlocks = ((int64_t)1 << 32) / 256 - 1;

// Workgroups of a norm's reverse mode over this many rows at most: each sums the
// weight gradients of its rows and writes one partial row, which a second launch
// adds in a fixed order.  And the bytes of its workspace with `weights` weights.
int norm_bwd_blocks(int64_t rows, int32_t dim);
size_t norm_bwd_workspace_bytes(int64_t rows, int32_t dim, int weights);

flare_status check_io(int32_t io_dtype);
flare_status check_eps(float eps);
flare_status check_gate(const void *gate, int32_t activation, int64_t stride, int64_t row);
flare_status check_gated_norm(int64_t tokens, int32_t heads, int32_t dim, int32_t io_dtype, const void *x,
                              int64_t x_stride, const void *gate, int64_t gate_stride, const float *weight,
                              int32_t activation);
flare_status check_residual_norm(int64_t tokens, int32_t dim, int32_t io_dtype, int32_t res_dtype, const void *x,
                                 int64_t x_stride, const void *residual, const void *gate, int64_t gate_stride,
                                 const float *w_pre, int32_t activation);
flare_status check_workspace(const void *workspace, size_t bytes, size_t need);
flare_status check_rotary(int64_t tokens, const flare_rotary_shape *s, const int32_t *positions, const double *freqs,
                          const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *q_out);
// the launch's limit, once the arguments are laid out
flare_status check_rotary_blocks(const RotaryArgs &a);
flare_status check_qk_norm(const QkNormArgs &a, int64_t tokens);
int64_t qk_norm_bwd_blocks(int64_t tokens);
size_t qk_norm_bwd_workspace_bytes(int64_t tokens, int32_t dim);
// a cache's sizes and pointers; `what` names the call
flare_status check_cache4(const char *what, int32_t dim, int64_t num_pages, int32_t page, const Cache4 &k, const Cache4 &v);
flare_status check_step_tables(const StepTablesArgs &a);
// shape alone (for the size query), then everything
flare_status check_attention_shape(int32_t num_req, const flare_attention_shape *s, int32_t max_seq_len,
                                   int32_t prefix_len);
flare_status check_attention_fp4_shape(int32_t num_req, const flare_attention_shape *s, int32_t max_seq_len,
                                       int32_t prefix_len);
flare_status check_attention_fp4_cache(const BlockAttnArgs &a, int64_t num_pages);
BlockAttnArgs attention_args(int32_t num_req, const flare_attention_shape *s, int32_t max_seq_len,
                             int32_t prefix_len);

}  // namespace flare
