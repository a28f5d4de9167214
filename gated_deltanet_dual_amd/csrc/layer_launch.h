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
hipError_t launch_step_tables(const StepTablesArgs &a, hipStream_t st);
hipError_t launch_block_attention(const BlockAttnArgs &a, const AttnPlan &p, hipStream_t st);

}  // namespace flare
