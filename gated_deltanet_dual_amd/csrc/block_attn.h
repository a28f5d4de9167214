// block_attn.h -- how a block attention is cut into parts (host and device;
// no HIP types, so that the workspace size can be told and tested without a GPU).
#pragma once

#include "layer_ops.h"

namespace flare {

// Workgroups come in octets, one for each XCD, and runs of 32 octets, one for each of
// an XCD's CUs.
constexpr int kOctets = 32;

struct AttnPlan {
  int prefix_tiles, own_tiles;  // 16-row query tiles of a wave (4 waves a workgroup)
  int page_shift;
  int merged;                   // a short prefix: every request passes it before its own keys
  int prefix_parts, prefix_chunk, prefix_groups;  // parts of the prefix, keys a part, row groups
  int own_parts, own_chunk, own_groups;
  int64_t prefix_blocks, own_blocks;              // prefix: a multiple of 8, some of them empty
  int prefix_runs, own_runs;                      // and how many runs each fills
};

// A request's own keys: never more than its table or the caller's bound holds.
FLARE_HD int attn_own_len(const BlockAttnArgs &a, int32_t len) {
  const int most = a.max_seq_len;
  return len < 0 ? 0 : len > most ? most : len;
}

// a.max_seq_len <= max_pages * page
AttnPlan attn_plan(const BlockAttnArgs &a);
// The workgroups that a plan launches: those of the prefix and of the own keys, each
// filled up to whole runs.
int64_t attn_launch_blocks(const AttnPlan &p);
size_t block_attention_workspace_bytes(const BlockAttnArgs &a, const AttnPlan &p);

}  // namespace flare
