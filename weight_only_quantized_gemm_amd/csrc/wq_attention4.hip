// How the attention over a 4-bit cache is cut, and its launch (wq_paged_attention4).
#include "wq_attention4_kernel.h"

namespace wq {

AttnPlan attn4_plan(int batch, int q_heads, int kv_heads, int head_dim, int group_size, int max_len,
                    int window) {
  const int groups = head_dim / group_size, group = q_heads / kv_heads;
  Columns c;
  const auto plan_of = [&](bool pairs) {
    c = columns_of(group, kv_heads, groups, head_dim, pairs);
    const int heads = 1 << c.heads_log2;
    AttnPlan plan{};
    plan.block_shift = c.heads_log2;
    plan.head_blocks = (c.kv_heads * group + heads - 1) / heads;
    plan.units = (kv_heads + c.kv_heads - 1) / c.kv_heads * plan.head_blocks;
    return plan;
  };
  // Positions a sequence may need, from the tile that holds the window's first.  Short sequences stay
  // whole, by single KV heads, which makes more work-groups and leaves out the join; the longer ones
  // may be, the more work-groups they make (us of 32 heads over 8 of 128, whole and cut: one of 1000
  // 12.9 and 11.4; 16 of up to 500 10.2 and 12.8, up to 1500 17.7 and 15.9; 32 up to 2000 22.5 and 23.3,
  // up to 2500 26.2 and 24.9; 64 up to 2000 28.7 and 31.5, up to 4000 46.6 and 43.5; 128 up to 2000
  // 50.8 and 47.9).
  AttnPlan plan = plan_of(false);
  const long span = window > 0 && window < max_len - 64 ? window + 63 : max_len;
  const long whole = std::max(672l, 9 * std::min(256l, (long)batch * plan.units));
  if (span <= whole) return plan;
  plan = plan_of(true);
  // Two work-groups a CU (us with 256, 512 and 768: 16 sequences of up to 4096 23.9, 23.0, 25.0; 64 of
  // 64 heads of up to 8192, groups of 32, 135, 102, 123; 16 of up to 4096, heads of 256, 41.7, 39.5,
  // 42.2).
  plan.ranges = std::max(1, 512 / plan.units);
  return plan;
}

size_t attn4_workspace_bytes(const AttnPlan& plan, int batch, int q_heads, int kv_heads,
                             int head_dim, int group_size) {
  const Columns c = columns_of(q_heads / kv_heads, kv_heads, head_dim / group_size, head_dim,
                               plan.ranges > 0);
  // (as many rows to a partial as a work-group has heads)
  return attn_workspace_bytes(plan, batch, c.kv_heads * (q_heads / kv_heads), 1, head_dim);
}

hipError_t launch_paged_attention4(const wq_attn4_args& a, const AttnPlan& plan,
                                   hipStream_t stream) {
  const int group = a.q_heads / a.cache.kv_heads, groups = a.cache.head_dim / a.pairs.group_size;
  const Columns c = columns_of(group, a.cache.kv_heads, groups, a.cache.head_dim, plan.ranges > 0);
  Attn4Args p{};
  // the query heads of a work-group's KV heads count as one's
  static_cast<AttnArgs&>(p) = attn_args(a, plan, c.kv_heads * group);
  p.kv_group = group;
  p.k_pairs = static_cast<const uint32_t*>(a.pairs.k);
  p.v_pairs = static_cast<const uint32_t*>(a.pairs.v);
  p.pair_page = a.pairs.page_stride;
  p.pair_slot = a.pairs.slot_stride;
  p.pair_head = a.pairs.head_stride;
  p.group_size = a.pairs.group_size;
  const int64_t limit = int64_t(1) << 32;
  p.short_strides = p.page_stride < limit && p.page_size * p.slot_stride < limit &&
                    p.pair_page < limit && p.page_size * p.pair_slot < limit;
  const bool bf16 = (a.flags & WQ_FLAG_BF16) != 0;
  // units that read the same rows or share lines, of codes or of pairs, as in the 16-bit kernel
  const auto shares = [&](int64_t head, int64_t slot) { return head < slot && head % 128 != 0; };
  p.near_units =
      plan.head_blocks > 1 ||
      (plan.units > 1 && (shares(c.kv_heads * p.head_stride / 2, p.slot_stride / 2) ||
                          shares(c.kv_heads * p.pair_head * 4, p.pair_slot * 4)));
  const dim3 grid = attn_grid(p);
  const hipError_t e = (bf16 ? launch_attn4_bf16 : launch_attn4_fp16)(p, c, grid, stream);
  if (e != hipSuccess || plan.ranges == 0) return e;
  switch (plan.block_shift) {
    case 1: return launch_attn_join<1>(p, bf16, stream);
    case 2: return launch_attn_join<2>(p, bf16, stream);
    case 3: return launch_attn_join<3>(p, bf16, stream);
    case 4: return launch_attn_join<4>(p, bf16, stream);
    case 5: return launch_attn_join<5>(p, bf16, stream);
  }
  return hipErrorNotSupported;
}

}  // namespace wq
