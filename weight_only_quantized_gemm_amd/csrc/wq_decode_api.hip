// C ABI of the decode-step operators: argument validation and launches (see include/wq.h).
#include <algorithm>
#include <limits>

#include "wq.h"
#include "wq_decode.h"
#include "wq_internal.h"

namespace {

int fail(int stage, int code) { return WQ_STATUS(stage, code); }
int shape_error() { return fail(WQ_STAGE_SHAPE, WQ_ERR_SHAPE); }
int flags_error() { return fail(WQ_STAGE_ARGS, WQ_ERR_FLAGS); }

int launched(hipError_t e) { return e == hipSuccess ? 0 : fail(WQ_STAGE_LAUNCH, (int)e); }

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int check_ptr(const void* p, size_t align) {
  if (p == nullptr) return fail(WQ_STAGE_ARGS, WQ_ERR_NULL);
  return aligned(p, align) ? 0 : fail(WQ_STAGE_ARGS, WQ_ERR_ALIGN);
}

int check_optional(const void* p, size_t align) {
  return p == nullptr || aligned(p, align) ? 0 : fail(WQ_STAGE_ARGS, WQ_ERR_ALIGN);
}

template <class Args>
int check_abi(const Args* a) {
  if (a == nullptr) return fail(WQ_STAGE_ARGS, WQ_ERR_NULL);
  if (a->abi_version != WQ_ABI_VERSION || a->struct_size != sizeof(Args) || a->reserved != 0)
    return fail(WQ_STAGE_ARGS, WQ_ERR_ABI);
  return 0;
}

bool row_stride_ok(int ld, int64_t least) { return ld >= least && ld % 8 == 0; }

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

constexpr int kMaxHeads = 65535;  // heads of one kind: grid axes and 32-bit row offsets
constexpr int kMaxRows = (1 << 22) - 1;     // 1024 threads each, below 2^32 in a launch
constexpr int kMaxTokens = (1 << 24) - 1;   // 256 threads each

int check_cache(const wq_kv_cache& c, uint32_t flags) {
  const bool fp8 = (flags & WQ_FLAG_FP8) != 0;
  if (c.num_pages < 1 || c.page_size < 1 || c.kv_heads < 1 || c.kv_heads > kMaxHeads ||
      c.head_dim < 16 || c.head_dim > 256 || c.head_dim % 8 != 0)
    return shape_error();
  const int64_t strides[3] = {c.page_stride, c.slot_stride, c.head_stride};
  const int64_t counts[3] = {c.num_pages, c.page_size, c.kv_heads};
  int64_t extent = c.head_dim;
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < 0 || strides[i] % 8 != 0 || (counts[i] > 1 && strides[i] < c.head_dim))
      return shape_error();
    if (counts[i] > 1 && strides[i] > (std::numeric_limits<int64_t>::max() / 8) / counts[i])
      return fail(WQ_STAGE_SHAPE, WQ_ERR_OVERFLOW);
    extent += strides[i] * (counts[i] - 1);
    if (extent > std::numeric_limits<int64_t>::max() / 8)
      return fail(WQ_STAGE_SHAPE, WQ_ERR_OVERFLOW);
  }
  int st;
  if ((st = check_ptr(c.k, fp8 ? 8 : 16)) || (st = check_ptr(c.v, fp8 ? 8 : 16))) return st;
  if (!fp8 && (c.k_scale != nullptr || c.v_scale != nullptr)) return flags_error();
  if ((st = check_optional(c.k_scale, 4)) || (st = check_optional(c.v_scale, 4))) return st;
  return 0;
}

}  // namespace

extern "C" {

int wq_add_rms_norm(const wq_norm_args* args) {
  int st = check_abi(args);
  if (st) return st;
  const wq_norm_args& a = *args;
  if (a.flags & ~(uint32_t)WQ_FLAG_BF16) return flags_error();
  if (a.rows < 1 || a.rows > kMaxRows || a.n < 8 || a.n > 65536 || a.n % 8 != 0 ||
      !(a.eps >= 0.f) || !row_stride_ok(a.ldx, a.n) || !row_stride_ok(a.ldy, a.n) ||
      (a.delta != nullptr && !row_stride_ok(a.ldd, a.n)) ||
      (a.sum_out != nullptr && !row_stride_ok(a.lds, a.n)))
    return shape_error();
  if ((st = check_ptr(a.x, 16)) || (st = check_ptr(a.weight, 16)) || (st = check_ptr(a.y, 16)) ||
      (st = check_optional(a.delta, 16)) || (st = check_optional(a.sum_out, 16)))
    return st;
  // a sum is written only where there is one, and not over the normalized row
  if (a.sum_out != nullptr && (a.delta == nullptr || a.sum_out == a.y)) return flags_error();
  return launched(wq::launch_add_rms_norm(a, as_stream(a.stream)));
}

int wq_rope_append(const wq_rope_args* args) {
  int st = check_abi(args);
  if (st) return st;
  const wq_rope_args& a = *args;
  if (a.flags & ~(uint32_t)(WQ_FLAG_BF16 | WQ_FLAG_FP8)) return flags_error();
  if (a.interleaved != 0 && a.interleaved != 1) return flags_error();
  if ((st = check_cache(a.cache, a.flags))) return st;
  const int64_t d = a.cache.head_dim;
  if (a.tokens < 1 || a.tokens > kMaxTokens || a.q_heads < 0 || a.q_heads > kMaxHeads ||
      a.rot_dim < 0 || a.rot_dim > d || a.rot_dim % 8 != 0 || a.axes < 1 ||
      a.axes > WQ_MAX_ROPE_AXES)
    return shape_error();
  if (!row_stride_ok(a.ldk, a.cache.kv_heads * d) || !row_stride_ok(a.ldv, a.cache.kv_heads * d) ||
      (a.q_heads > 0 &&
       (!row_stride_ok(a.ldq, a.q_heads * d) || !row_stride_ok(a.ldqo, a.q_heads * d))))
    return shape_error();
  int64_t pairs = 0;
  for (int i = 0; i < a.axes; ++i) {
    if (a.sections[i] < 0) return shape_error();
    pairs += a.sections[i];
  }
  if (pairs != a.rot_dim / 2) return shape_error();
  if ((st = check_ptr(a.k, 16)) || (st = check_ptr(a.v, 16)) || (st = check_ptr(a.slots, 8)))
    return st;
  if (a.q_heads > 0 && ((st = check_ptr(a.q, 16)) || (st = check_ptr(a.q_out, 16)))) return st;
  if (a.rot_dim > 0 && ((st = check_ptr(a.positions, 4)) || (st = check_ptr(a.inv_freq, 4))))
    return st;
  return launched(wq::launch_rope_append(a, as_stream(a.stream)));
}

int wq_paged_attention_workspace_bytes(int batch, int q_heads, int kv_heads, int head_dim,
                                       int max_len, int window, uint32_t flags,
                                       size_t* bytes_out) {
  if (bytes_out == nullptr) return fail(WQ_STAGE_ARGS, WQ_ERR_NULL);
  if (flags & ~(uint32_t)(WQ_FLAG_BF16 | WQ_FLAG_FP8)) return flags_error();
  if (batch < 1 || batch > kMaxHeads || kv_heads < 1 || q_heads < kv_heads ||
      q_heads > kMaxHeads || q_heads % kv_heads != 0 || head_dim < 16 || head_dim > 256 ||
      head_dim % 8 != 0 || max_len < 1 || max_len > (1 << 30) || window < 0)
    return shape_error();
  const wq::AttnPlan plan = wq::attn_plan(batch, q_heads, kv_heads, head_dim, max_len, window,
                                          (flags & WQ_FLAG_FP8) != 0);
  // work-groups of one launch; steps of 128 positions over all sequences, counted in 32 bits
  const int64_t steps = (window > 0 ? std::min(window, max_len) : max_len) / 128 + 2;
  if ((int64_t)(plan.ranges > 0 ? plan.ranges : batch) * plan.units > (1 << 23) ||
      batch * steps > (1 << 30))
    return fail(WQ_STAGE_SHAPE, WQ_ERR_OVERFLOW);
  *bytes_out = wq::attn_workspace_bytes(plan, batch, q_heads, kv_heads, head_dim);
  return 0;
}

int wq_paged_attention(const wq_attn_args* args) {
  int st = check_abi(args);
  if (st) return st;
  const wq_attn_args& a = *args;
  if (a.flags & ~(uint32_t)(WQ_FLAG_BF16 | WQ_FLAG_FP8)) return flags_error();
  if ((st = check_cache(a.cache, a.flags))) return st;
  size_t need = 0;
  if ((st = wq_paged_attention_workspace_bytes(a.batch, a.q_heads, a.cache.kv_heads,
                                               a.cache.head_dim, a.max_len, a.window, a.flags,
                                               &need)))
    return st;
  const int64_t row = (int64_t)a.q_heads * a.cache.head_dim;
  if (!row_stride_ok(a.ldq, row) || !row_stride_ok(a.ldo, row) || a.table_stride < 1 ||
      (int64_t)a.table_stride * a.cache.page_size < a.max_len ||
      (a.keep != nullptr && a.keep_stride < a.max_len))
    return shape_error();
  // a scale or cap that is no number would make every output one
  if (!(a.scale - a.scale == 0.f) || !(a.softcap >= 0.f && a.softcap - a.softcap == 0.f))
    return shape_error();
  if ((st = check_ptr(a.q, 16)) || (st = check_ptr(a.out, 16)) || (st = check_optional(a.lse, 4)) ||
      (st = check_ptr(a.block_table, 4)) || (st = check_ptr(a.lens, 4)))
    return st;
  if (need > 0) {
    if (a.workspace == nullptr || a.workspace_bytes < need)
      return fail(WQ_STAGE_ARGS, WQ_ERR_WORKSPACE);
    if (!aligned(a.workspace, 16)) return fail(WQ_STAGE_ARGS, WQ_ERR_ALIGN);
  }
  const wq::AttnPlan plan = wq::attn_plan(a.batch, a.q_heads, a.cache.kv_heads, a.cache.head_dim,
                                          a.max_len, a.window, (a.flags & WQ_FLAG_FP8) != 0);
  return launched(wq::launch_paged_attention(a, plan, as_stream(a.stream)));
}

int wq_moe_layer_workspace_bytes(int tokens, int n_expert, int top_k, int hidden, int inter,
                                 size_t* bytes_out) {
  if (bytes_out == nullptr) return fail(WQ_STAGE_ARGS, WQ_ERR_NULL);
  if (tokens < 1 || tokens > WQ_MOE_MAX_TOKENS || n_expert < 1 || n_expert > WQ_MOE_MAX_EXPERTS ||
      top_k < 1 || top_k > n_expert || top_k > WQ_MOE_MAX_TOPK || hidden < 256 ||
      hidden % 256 != 0 || inter < 128 || inter % 128 != 0)
    return shape_error();
  // the chunk counts of a wave's offsets stay within 32 bits
  if ((int64_t)hidden * inter / 2 > (int64_t)std::numeric_limits<int32_t>::max())
    return fail(WQ_STAGE_SHAPE, WQ_ERR_OVERFLOW);
  *bytes_out = wq::moe_workspace_bytes(tokens, n_expert, top_k, hidden, inter);
  return 0;
}

static int check_bank(const wq_expert_bank& b, int64_t k, int64_t n, uint32_t flags) {
  if (b.reserved != 0) return fail(WQ_STAGE_ARGS, WQ_ERR_ABI);
  const bool fp8 = (flags & WQ_FLAG_FP8) != 0, zp = (flags & WQ_FLAG_HAS_ZP) != 0;
  if (b.group_size != -1 && (b.group_size <= 0 || b.group_size % 16 != 0 || k % b.group_size != 0))
    return shape_error();
  if (fp8 && b.group_size != -1 && b.group_size != 128) return shape_error();
  if (zp != (b.zp != nullptr)) return flags_error();
  int st;
  if ((st = check_ptr(b.b, 16)) || (st = check_ptr(b.s, 16)) || (zp && (st = check_ptr(b.zp, 16))))
    return st;
  const int64_t units = k / wq::scale_unit_rows((int)k, b.group_size);
  if (b.b_stride_bytes < (size_t)(fp8 ? k * n : k * n / 2) || b.b_stride_bytes % 16 ||
      b.s_stride_bytes < (size_t)(units * n * 2) || b.s_stride_bytes % 16 ||
      (zp && (b.zp_stride_bytes < (size_t)(units * n / 2) || b.zp_stride_bytes % 16)))
    return shape_error();
  return 0;
}

int wq_moe_layer(const wq_moe_args* args) {
  int st = check_abi(args);
  if (st) return st;
  const wq_moe_args& a = *args;
  if (a.flags & ~(uint32_t)(WQ_FLAG_BF16 | WQ_FLAG_FP8 | WQ_FLAG_HAS_ZP)) return flags_error();
  if ((a.flags & WQ_FLAG_FP8) && (a.flags & WQ_FLAG_HAS_ZP)) return flags_error();
  if (a.renormalize != 0 && a.renormalize != 1) return flags_error();
  size_t need = 0;
  if ((st = wq_moe_layer_workspace_bytes(a.tokens, a.n_expert, a.top_k, a.hidden, a.inter, &need)))
    return st;
  if (!row_stride_ok(a.ldx, a.hidden) || !row_stride_ok(a.ldy, a.hidden) ||
      (a.residual != nullptr && !row_stride_ok(a.ldr, a.hidden)))
    return shape_error();
  if ((st = check_ptr(a.x, 16)) || (st = check_ptr(a.router, 16)) || (st = check_ptr(a.y, 16)) ||
      (st = check_optional(a.residual, 16)) || (st = check_optional(a.ids, 4)) ||
      (st = check_optional(a.weights, 4)))
    return st;
  if ((st = check_bank(a.gate_up, a.hidden, 2 * (int64_t)a.inter, a.flags)) ||
      (st = check_bank(a.down, a.inter, a.hidden, a.flags)))
    return st;
  if (a.workspace == nullptr || a.workspace_bytes < need)
    return fail(WQ_STAGE_ARGS, WQ_ERR_WORKSPACE);
  if (!aligned(a.workspace, 16)) return fail(WQ_STAGE_ARGS, WQ_ERR_ALIGN);
  const int gu = 128 / wq::scale_unit_rows(a.hidden, a.gate_up.group_size);
  const int dn = 128 / wq::scale_unit_rows(a.inter, a.down.group_size);
  return launched(wq::launch_moe_layer(a, gu, dn, as_stream(a.stream)));
}

}  // extern "C"
