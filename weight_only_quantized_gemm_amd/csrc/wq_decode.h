// Host-side launchers of the decode-step kernels (norm, rotary append, paged attention, MoE
// layer), shared between the kernel files and the C ABI layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "wq.h"

namespace wq {

hipError_t launch_add_rms_norm(const wq_norm_args& a, hipStream_t stream);

hipError_t launch_rope_append(const wq_rope_args& a, hipStream_t stream);

hipError_t launch_norm_rope_append(const wq_norm_rope_args& a, hipStream_t stream);
hipError_t launch_cache4_read(const wq_cache4_read_args& a, hipStream_t stream);

// How a call's positions are cut: at most `ranges` ranges of equal length over all sequences
// (0: one range for each sequence), each taken by `units` work-groups, one per KV head and
// block of 2^block_shift of its query heads.  Sequences that no range holds whole leave fp32 partials
// that a second kernel joins.
struct AttnPlan {
  int ranges;
  int units;
  int head_blocks;  // blocks of query heads per KV head
  int block_shift;  // 2^block_shift query heads to a block
};
AttnPlan attn_plan(int batch, int q_heads, int kv_heads, int head_dim, int max_len, int window,
                   bool kv8);
size_t attn_workspace_bytes(const AttnPlan& plan, int batch, int q_heads, int kv_heads,
                            int head_dim);
hipError_t launch_paged_attention(const wq_attn_args& a, const AttnPlan& plan,
                                  hipStream_t stream);


AttnPlan attn4_plan(int batch, int q_heads, int kv_heads, int head_dim, int group_size, int max_len,
                    int window);
size_t attn4_workspace_bytes(const AttnPlan& plan, int batch, int q_heads, int kv_heads,
                             int head_dim, int group_size);
hipError_t launch_paged_attention4(const wq_attn4_args& a, const AttnPlan& plan,
                                   hipStream_t stream);

size_t sample_workspace_bytes(int rows, int vocab, uint32_t flags);
hipError_t launch_sample(const wq_sample_args& a, hipStream_t stream);

size_t moe_workspace_bytes(int tokens, int n_expert, int top_k, int hidden, int inter);
// gpc: scale units per 128 rows of K of each bank (1, 2, 4 or 8).
hipError_t launch_moe_layer(const wq_moe_args& a, int gate_up_gpc, int down_gpc,
                            hipStream_t stream);

}  // namespace wq
