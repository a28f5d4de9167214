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
flare_status check_step_tables(const StepTablesArgs &a);
// shape alone (for the size query), then everything
flare_status check_attention_shape(int32_t num_req, const flare_attention_shape *s, int32_t max_seq_len,
                                   int32_t prefix_len);
BlockAttnArgs attention_args(int32_t num_req, const flare_attention_shape *s, int32_t max_seq_len,
                             int32_t prefix_len);

}  // namespace flare
