// api_layer.hip -- extern "C" entry points of the operators around the GDN step
// (norms, rotary positions, serving-step tables, block attention).  As in
// api.hip: everything is validated on the host before anything is enqueued, and
// nothing is allocated, freed or synchronised.
#include <hip/hip_runtime.h>

#include "block_attn.h"
#include "host_plan.h"
#include "layer_launch.h"

using namespace flare;

static flare_status hip_status(hipError_t e, const char *what) {
  if (e == hipSuccess) return FLARE_OK;
  return fail(FLARE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

extern "C" {

flare_status flare_gated_norm(int64_t tokens, int32_t heads, int32_t dim, int32_t io_dtype, const void *x,
                              int64_t x_stride, const void *gate, int64_t gate_stride, const float *weight,
                              int32_t activation, float eps, void *y, float *rstd, void *stream) {
  clear_error();
  flare_status st = check_gated_norm(tokens, heads, dim, io_dtype, x, x_stride, gate, gate_stride, weight, activation);
  if (st == FLARE_OK) st = check_eps(eps);
  if (st != FLARE_OK) return st;
  if (tokens == 0) return FLARE_OK;
  if (!y) return fail(FLARE_ERR_NULL, "gated_norm: y is NULL");
  GatedNormArgs a{};
  a.tokens = tokens;
  a.heads = heads;
  a.dim = dim;
  a.bf16 = io_dtype == FLARE_BF16;
  a.act = gate ? activation : -1;
  a.eps = eps;
  a.x = x; a.gate = gate; a.x_stride = x_stride; a.gate_stride = gate_stride;
  a.weight = weight; a.y = y; a.rstd = rstd;
  return hip_status(launch_gated_norm(a, (hipStream_t)stream), "gated_norm launch");
}

size_t flare_gated_norm_bwd_workspace_size(int64_t tokens, int32_t heads, int32_t dim) {
  if (tokens < 0 || tokens > INT32_MAX || heads < 1 || dim < 1 || dim > 16384 || tokens * heads > INT32_MAX) return 0;
  return norm_bwd_workspace_bytes(tokens * heads, dim, 1);
}

flare_status flare_gated_norm_bwd(int64_t tokens, int32_t heads, int32_t dim, int32_t io_dtype, const void *x,
                                  int64_t x_stride, const void *gate, int64_t gate_stride, const float *weight,
                                  int32_t activation, const float *rstd, const void *dy, int64_t dy_stride, void *dx,
                                  void *dgate, float *dweight, void *workspace, size_t workspace_bytes, void *stream) {
  clear_error();
  flare_status st = check_gated_norm(tokens, heads, dim, io_dtype, x, x_stride, gate, gate_stride, weight, activation);
  if (st != FLARE_OK) return st;
  if (dy_stride < (int64_t)heads * dim) return fail(FLARE_ERR_SHAPE, "dy_stride below a row");
  if (!dweight || (tokens > 0 && (!rstd || !dy || !dx || (gate && !dgate))))
    return fail(FLARE_ERR_NULL, "gated_norm_bwd: a required pointer is NULL");
  st = check_workspace(workspace, workspace_bytes, norm_bwd_workspace_bytes(tokens * heads, dim, 1));
  if (st != FLARE_OK) return st;
  GatedNormArgs a{};
  a.tokens = tokens;
  a.heads = heads;
  a.dim = dim;
  a.bf16 = io_dtype == FLARE_BF16;
  a.act = gate ? activation : -1;
  a.x = x; a.gate = gate; a.dy = dy;
  a.x_stride = x_stride; a.gate_stride = gate_stride; a.dy_stride = dy_stride;
  a.weight = weight; a.rstd = const_cast<float *>(rstd);
  a.dx = dx; a.dgate = dgate; a.dweight = dweight;
  a.part = reinterpret_cast<float *>(workspace);
  return hip_status(launch_gated_norm_bwd(a, (hipStream_t)stream), "gated_norm_bwd launch");
}

flare_status flare_residual_norm(int64_t tokens, int32_t dim, int32_t io_dtype, int32_t res_dtype, const void *x,
                                 int64_t x_stride, const void *residual, const void *gate, int64_t gate_stride,
                                 const float *w_pre, const float *w_post, const float *scale, int32_t activation,
                                 float eps, void *h, void *y, float *rstd, void *stream) {
  clear_error();
  flare_status st = check_residual_norm(tokens, dim, io_dtype, res_dtype, x, x_stride, residual, gate, gate_stride,
                                        w_pre, activation);
  if (st == FLARE_OK) st = check_eps(eps);
  if (st != FLARE_OK) return st;
  if (tokens == 0) return FLARE_OK;
  if (!h || !y) return fail(FLARE_ERR_NULL, "residual_norm: h or y is NULL");
  ResidualNormArgs a{};
  a.tokens = tokens;
  a.dim = dim;
  a.bf16 = io_dtype == FLARE_BF16;
  a.res_bf16 = res_dtype == FLARE_BF16;
  a.act = gate ? activation : -1;
  a.eps = eps;
  a.x = x; a.residual = residual; a.gate = gate;
  a.x_stride = x_stride; a.gate_stride = gate_stride;
  a.w_pre = w_pre; a.w_post = w_post; a.scale = scale;
  a.h = h; a.y = y; a.rstd = rstd;
  return hip_status(launch_residual_norm(a, (hipStream_t)stream), "residual_norm launch");
}

size_t flare_residual_norm_bwd_workspace_size(int64_t tokens, int32_t dim) {
  if (tokens < 0 || tokens > INT32_MAX || dim < 1 || dim > 16384) return 0;
  return norm_bwd_workspace_bytes(tokens, dim, 3);
}

flare_status flare_residual_norm_bwd(int64_t tokens, int32_t dim, int32_t io_dtype, int32_t res_dtype, const void *x,
                                     int64_t x_stride, const void *residual, const void *gate, int64_t gate_stride,
                                     const float *w_pre, const float *w_post, const float *scale, int32_t activation,
                                     const float *rstd, const void *dy, const void *dh, void *dx, void *dresidual,
                                     void *dgate, float *dw_pre, float *dw_post, float *dscale, void *workspace,
                                     size_t workspace_bytes, void *stream) {
  clear_error();
  flare_status st = check_residual_norm(tokens, dim, io_dtype, res_dtype, x, x_stride, residual, gate, gate_stride,
                                        w_pre, activation);
  if (st != FLARE_OK) return st;
  if (!dw_pre || (w_post && !dw_post) || (scale && !dscale) ||
      (tokens > 0 && (!rstd || !dy || !dx || !dresidual || (gate && !dgate))))
    return fail(FLARE_ERR_NULL, "residual_norm_bwd: a required pointer is NULL");
  st = check_workspace(workspace, workspace_bytes, norm_bwd_workspace_bytes(tokens, dim, 3));
  if (st != FLARE_OK) return st;
  ResidualNormArgs a{};
  a.tokens = tokens;
  a.dim = dim;
  a.bf16 = io_dtype == FLARE_BF16;
  a.res_bf16 = res_dtype == FLARE_BF16;
  a.act = gate ? activation : -1;
  a.x = x; a.residual = residual; a.gate = gate; a.dy = dy; a.dh = dh;
  a.x_stride = x_stride; a.gate_stride = gate_stride;
  a.w_pre = w_pre; a.w_post = w_post; a.scale = scale;
  a.rstd = const_cast<float *>(rstd);
  a.dx = dx; a.dres = dresidual; a.dgate = dgate;
  a.dw_pre = dw_pre; a.dw_post = dw_post; a.dscale = dscale;
  a.part[0] = reinterpret_cast<float *>(workspace);
  return hip_status(launch_residual_norm_bwd(a, (hipStream_t)stream), "residual_norm_bwd launch");
}

static RotaryArgs rotary_args(int64_t tokens, const flare_rotary_shape *s, const int32_t *positions,
                              const double *freqs, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                              void *q_out) {
  RotaryArgs a{};
  a.tokens = tokens;
  a.q_heads = s->q_heads;
  a.k_heads = s->k_heads;
  a.dim = s->dim;
  a.half = s->half;
  a.bf16 = s->io_dtype == FLARE_BF16;
  a.interleaved = s->interleaved;
  a.mscale = s->mscale;
  a.sign = 1.0f;
  a.positions = positions;
  a.freqs = freqs;
  a.q = q; a.k = k; a.q_stride = q_stride; a.k_stride = k_stride;
  a.q_out = q_out;
  return a;
}

flare_status flare_rotary(int64_t tokens, const flare_rotary_shape *shape, const int32_t *positions,
                          const double *freqs, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                          int32_t inverse, void *q_out, void *k_out, void *stream) {
  clear_error();
  flare_status st = check_rotary(tokens, shape, positions, freqs, q, q_stride, k, k_stride, q_out);
  if (st != FLARE_OK) return st;
  if (inverse != 0 && inverse != 1) return fail(FLARE_ERR_UNSUPPORTED, "rotary: inverse %d unknown", inverse);
  if (tokens > 0 && shape->k_heads > 0 && !k_out) return fail(FLARE_ERR_NULL, "rotary: k_out is NULL");
  RotaryArgs a = rotary_args(tokens, shape, positions, freqs, q, q_stride, k, k_stride, q_out);
  if (inverse) a.sign = -1.0f;
  a.k_out = k_out;
  st = check_rotary_blocks(a);
  if (st != FLARE_OK) return st;
  return hip_status(launch_rotary(a, (hipStream_t)stream), "rotary launch");
}

flare_status flare_rotary_cache(int64_t tokens, const flare_rotary_shape *shape, const int32_t *positions,
                                const double *freqs, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                const void *v, int64_t v_stride, const int64_t *slots, void *q_out, void *k_cache,
                                void *v_cache, int64_t num_pages, int32_t page, void *stream) {
  clear_error();
  flare_status st = check_rotary(tokens, shape, positions, freqs, q, q_stride, k, k_stride, q_out);
  if (st != FLARE_OK) return st;
  if (shape->k_heads < 1) return fail(FLARE_ERR_SHAPE, "rotary_cache: no k heads");
  if (page < 1 || num_pages < 0 || num_pages > INT32_MAX) return fail(FLARE_ERR_SHAPE, "rotary_cache: page or num_pages");
  if (v_stride < (int64_t)shape->k_heads * shape->dim) return fail(FLARE_ERR_SHAPE, "rotary_cache: v_stride below a row");
  if (tokens > 0 && (!v || !slots || (num_pages > 0 && (!k_cache || !v_cache))))
    return fail(FLARE_ERR_NULL, "rotary_cache: a required pointer is NULL");
  RotaryArgs a = rotary_args(tokens, shape, positions, freqs, q, q_stride, k, k_stride, q_out);
  a.v = v;
  a.v_stride = v_stride;
  a.slots = slots;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.num_pages = num_pages;
  a.page = page;
  st = check_rotary_blocks(a);
  if (st != FLARE_OK) return st;
  return hip_status(launch_rotary(a, (hipStream_t)stream), "rotary_cache launch");
}

flare_status flare_step_tables(int32_t num_req, const int32_t *seq_lens, const int32_t *new_lens, int32_t *block_table,
                               int32_t max_pages, const int32_t *free_pages, int64_t num_free,
                               const int32_t *pages_used, int32_t page, int32_t position_offset, int64_t max_tokens,
                               int32_t *cu_new, int32_t *positions, int64_t *slots, int32_t *seq_lens_out,
                               int32_t *pages_used_out, int32_t *status, void *stream) {
  clear_error();
  StepTablesArgs a{};
  a.num_req = num_req;
  a.max_pages = max_pages;
  a.page = page;
  a.num_free = num_free;
  a.max_tokens = max_tokens;
  a.position_offset = position_offset;
  a.seq_lens = seq_lens; a.new_lens = new_lens; a.free_pages = free_pages; a.pages_used = pages_used;
  a.block_table = block_table; a.cu_new = cu_new; a.positions = positions; a.slots = slots;
  a.seq_lens_out = seq_lens_out; a.pages_used_out = pages_used_out; a.status = status;
  const flare_status st = check_step_tables(a);
  if (st != FLARE_OK) return st;
  return hip_status(launch_step_tables(a, (hipStream_t)stream), "step_tables launch");
}

size_t flare_block_attention_workspace_size(int32_t num_req, const flare_attention_shape *shape, int32_t max_seq_len,
                                            int32_t prefix_len) {
  if (check_attention_shape(num_req, shape, max_seq_len, prefix_len) != FLARE_OK) return 0;
  const BlockAttnArgs a = attention_args(num_req, shape, max_seq_len, prefix_len);
  return block_attention_workspace_bytes(a, attn_plan(a));
}

flare_status flare_block_attention(int32_t num_req, const flare_attention_shape *shape, const void *q,
                                   const void *k_cache, const void *v_cache, int64_t num_pages,
                                   const int32_t *block_table, int32_t max_pages, const int32_t *seq_lens,
                                   int32_t max_seq_len, const int32_t *prefix_table, int32_t prefix_len, void *o,
                                   float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  clear_error();
  flare_status st = check_attention_shape(num_req, shape, max_seq_len, prefix_len);
  if (st != FLARE_OK) return st;
  if (num_pages < 0 || num_pages > INT32_MAX || max_pages < 0)
    return fail(FLARE_ERR_SHAPE, "block_attention: num_pages or max_pages");
  if (max_seq_len > (int64_t)max_pages * shape->page)
    return fail(FLARE_ERR_SHAPE, "block_attention: max_seq_len %d beyond the table's %d pages of %d", max_seq_len,
                max_pages, shape->page);
  if ((max_seq_len > 0 || prefix_len > 0) && num_pages == 0)
    return fail(FLARE_ERR_SHAPE, "block_attention: keys, but a cache of no pages");
  if (num_req == 0) return FLARE_OK;
  if (!q || !o || !seq_lens || (max_seq_len > 0 && !block_table) || (prefix_len > 0 && !prefix_table) ||
      (num_pages > 0 && (!k_cache || !v_cache)))
    return fail(FLARE_ERR_NULL, "block_attention: a required pointer is NULL");
  if ((((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)o) & 15u) != 0)
    return fail(FLARE_ERR_ALIGN, "block_attention: q, the caches and o must be 16-byte aligned");
  BlockAttnArgs a = attention_args(num_req, shape, max_seq_len, prefix_len);
  const AttnPlan p = attn_plan(a);
  const size_t need = block_attention_workspace_bytes(a, p);
  if (need > 0) {
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != FLARE_OK) return st;
  }
  if (attn_launch_blocks(p) > kMaxBlocks)
    return fail(FLARE_ERR_UNSUPPORTED, "block_attention: %lld workgroups, at most %lld", (long long)attn_launch_blocks(p),
                (long long)kMaxBlocks);
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
  a.block_table = block_table; a.seq_lens = seq_lens; a.prefix_table = prefix_table;
  a.o = o; a.lse = lse;
  a.part = reinterpret_cast<float *>(workspace);
  return hip_status(launch_block_attention(a, p, (hipStream_t)stream), "block_attention launch");
}

}  // extern "C"
