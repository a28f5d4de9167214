// layer_launch.h -- launchers of the operators around the GDN step (internal).
#pragma once

#include <hip/hip_runtime.h>

#include "block_attn.h"
#include "layer_ops.h"
#include "timing.h"

namespace flare {

hipError_t launch_gated_norm(const GatedNormArgs &a, hipStream_t st);
hipError_t launch_gated_norm_bwd(const GatedNormArgs &a, hipStream_t st);
hipError_t launch_residual_norm(const ResidualNormArgs &a, hipStream_t st);
hipError_t launch_residual_norm_bwd(const ResidualNormArgs &a, hipStream_t st);
hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st);
hipError_t launch_qk_norm_rotary(const QkNormArgs &a, hipStream_t st);
hipError_t launch_qk_norm_rotary_bwd(const QkNormArgs &a, hipStream_t st);
// out[i][c] = sum over b of part[i][b][c], i < 3, in a fixed order; out[i] NULL: left out
hipError_t launch_norm_partials(const float *part, int blocks, int dim, float *const (&out)[3], hipStream_t st);
hipError_t launch_cache_fp4_rows(const Cache4Rows &a, hipStream_t st);
hipError_t launch_step_tables(const StepTablesArgs &a, hipStream_t st);
// joins a call's parts; nothing where it has only one
hipError_t launch_attn_join(const BlockAttnArgs &a, const AttnPlan &p, hipStream_t st);
hipError_t launch_block_attention_fp4(const BlockAttnFp4Args &a, const AttnPlan &p, const AttnForms &f, hipStream_t st);
hipError_t launch_block_attention(const BlockAttnArgs &a, const AttnPlan &p, hipStream_t st);

}  // namespace flare
