// What the kernels of single-token attention over a paged cache share: their arguments, the cut of
// a batch's positions into ranges, and the join of a sequence's parts.
#pragma once

#include <algorithm>

#include "wq_decode.h"
#include "wq_device.h"
#include "wq_ranges.h"

namespace wq {

struct AttnArgs {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  const int32_t *table, *lens;
  const uint8_t* keep;
  // Partials of sequences that no range holds whole: [2 ranges][units][part_rows].
  float* part_o;   // [d], not divided by the sum
  float* part_ml;  // [2]: maximum (times log2 e) and sum
  int32_t* parts;  // [batch][2]: the ranges that hold a part of each sequence: first, count
  int64_t page_stride, slot_stride, head_stride;
  int num_pages, page_size, kv_heads, q_heads, d, group, head_blocks, max_len;
  int table_stride, keep_stride, ldq, ldo, window, batch;
  int units;       // work-groups of a range: KV heads times head blocks
  int part_rows;   // query heads of a partial: a work-group's most, or the group where it is smaller
  int ranges;      // most ranges that the batch is cut into; 0: one for each sequence
  int near_units;  // the units of a range share lines: they run on the same XCD
  uint32_t page_mul;  // position / page_size = umulhi(2 * position, page_mul) >> page_shift
  int page_shift;
  float scale, softcap;
};

namespace {

constexpr int kWaves = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Orders a wave's own LDS accesses (they execute in order; this keeps the compiler to it).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// c tanh(s / c) for x = s / c, within 10 2^-24 of its own value.  1 - 2 / (e^2x + 1) is off by
// some 2^-23 for any x, which is too much beside a small tanh (with a large c it is the score
// itself that is left); below 1/2 tanh(x) / x is a polynomial in x^2, fitted to 2^-26, times s.
// Both are formed, without branches (64 E4M3 sequences of up to 8192, capped: 87.5 us by the
// exponential alone, 92.6 so; 91.0 to 93.7, by the scores, with a branch round each exponential,
// and 89.6 to 96.4 with one for tiles of small scores.  Seven fp16 ones of up to 3001: 16.1; 16.4;
// 16.5 to 16.6; 16.5).
__device__ __forceinline__ float capped(float s, float x, float c) {
  const float z = x * x;
  float t = __builtin_fmaf(z, 0.017256992f, -0.053052951f);
  t = __builtin_fmaf(z, t, 0.13325988f);
  t = __builtin_fmaf(z, t, -0.33333150f);
  t = __builtin_fmaf(z, t, 1.f);
  const float e = __builtin_amdgcn_exp2f(2.f * kLog2e * x);
  const float large = c * (1.f - 2.f * __builtin_amdgcn_rcpf(e + 1.f)), small = s * t;
  return fabsf(x) < 0.5f ? small : large;
}

// Positions of a sequence that may be live start in the tile of the window's first one; they
// are dealt out in granules of a tile for each wave.
template <int TILE>
__device__ __forceinline__ int window_start(const AttnArgs& p, int len) {
  return p.window > 0 ? max(0, len - p.window) & ~(TILE - 1) : 0;
}
template <int TILE>
__device__ __forceinline__ int granules_of(const AttnArgs& p, int len) {
  return (len - window_start<TILE>(p, len) + kWaves * TILE - 1) / (kWaves * TILE);
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // row_shr 1, 2, 4, 8: each
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);  // row of 16 lanes
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast 15 to rows 1, 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // row_bcast 31 to rows 2, 3
  return x;
}

// A range's first sequence, the first of its granules there, and how many granules it has,
// over this and the next sequences.
struct Range {
  int b, first, left;
};

// The index-th range; false where it is empty.  All sequences' granules, one sequence after the
// other, are cut into `ranges` ranges of one length, the last ones shorter or empty.  The lengths
// are known only here, so every wave counts them, each lane a run of sequences.  (64 sequences of
// up to 8192 positions, E4M3: cut by the host by the longest length 135 us, in equal splits of
// each sequence 93.7, as here 88.8; unmasked 121.7 in equal splits, 112.5 here.)
template <int TILE>
__device__ __forceinline__ bool find_range(const AttnArgs& p, int index, bool publish, int lane,
                                           Range& out) {
  const int run = (p.batch + 63) / 64;
  const int b0 = lane * run, b1 = min(p.batch, b0 + run);
  const auto granules = [&](int b) {
    return granules_of<TILE>(p, max(0, min(p.lens[b], p.max_len)));
  };
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += granules(b);
  const int end = wave_scan(mine);
  const int total = __builtin_amdgcn_readlane(end, 63);
  const int chunk = range_length(total, p.ranges);
  if (publish) {  // where the join finds each sequence's parts
    int at = end - mine;
    for (int b = b0; b < b1; ++b) {
      const int n = granules(b);
      p.parts[2 * b] = at / chunk;
      p.parts[2 * b + 1] = n == 0 ? 0 : (at + n - 1) / chunk - at / chunk + 1;
      at += n;
    }
  }
  const int g0 = range_first(index, total, p.ranges);
  if (g0 < 0) return false;
  const int owner = __builtin_ctzll(__ballot(g0 < end));
  int at = __builtin_amdgcn_readlane(end - mine, owner);
  int b = owner * run;
  for (;; ++b) {
    const int n = granules(b);
    if (g0 < at + n) break;
    at += n;
  }
  out.b = b;
  out.first = g0 - at;
  out.left = min(chunk, total - g0);
  return true;
}

// Joins the parts of one query head: groups of threads, each d / 4 wide, take parts in turn
// and are added in group order.  Sequences of one part are done; empty ones become 0.  Bound by
// its launch and two trips to memory, the part numbers and the parts: 4.5 us for 16 sequences of
// 32 heads.  SHIFT: a work-group of the attention took up to 2^SHIFT query heads (as an argument
// of the kernel it cost the seven sequences above 0.25 us of 16.85: one more load before the others).
constexpr int kJoinThreads = 256;

template <bool BF16, int SHIFT>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs p) {
  using A = Act<BF16>;
  __shared__ f32x4 acc_lds[kJoinThreads];
  __shared__ float sum_lds[kJoinThreads], top_lds[kJoinThreads];
  const int head = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int first = p.parts[2 * b], parts = p.parts[2 * b + 1];
  if (parts == 1) return;  // the output is there
  const int64_t h = (int64_t)b * p.q_heads + head;
  const int per_row = p.d / 4;  // at most 64
  const int groups = kJoinThreads / per_row;
  const int g = tid / per_row, e = 4 * (tid - g * per_row);
  const int kvh = head / p.group, in_group = head - kvh * p.group;
  const int unit = kvh * p.head_blocks + (in_group >> SHIFT);
  const int64_t at = unit * p.part_rows + (in_group & ((1 << SHIFT) - 1));

  // each group of threads keeps its own maximum, so that no load waits for another split
  float top = -INFINITY, sum = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (g < groups) {
#pragma unroll 4
    for (int s = g; s < parts; s += groups) {
      // the second partial of the first range, then the first ones of the others
      const int64_t r = (2 * (int64_t)(first + s) + (s == 0)) * p.units * p.part_rows + at;
      const float ms = p.part_ml[2 * r], ls = p.part_ml[2 * r + 1];
      const f32x4 x = *reinterpret_cast<const f32x4*>(p.part_o + r * p.d + e);
      const float high = fmaxf(top, ms);
      const float ref = high == -INFINITY ? 0.f : high;
      const float fa = __builtin_amdgcn_exp2f(top - ref), fx = __builtin_amdgcn_exp2f(ms - ref);
      top = high;
      sum = sum * fa + ls * fx;
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = acc[c] * fa + x[c] * fx;
    }
  }
  acc_lds[tid] = acc;
  sum_lds[tid] = sum;
  top_lds[tid] = top;
  __syncthreads();
  if (g != 0) return;
  for (int k = 1; k < groups; ++k) top = fmaxf(top, top_lds[tid + k * per_row]);
  const float ref = top == -INFINITY ? 0.f : top;
  sum = 0.f;
  acc = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < groups; ++k) {
    const int at = tid + k * per_row;
    const float f = __builtin_amdgcn_exp2f(top_lds[at] - ref);
    sum = __builtin_fmaf(sum_lds[at], f, sum);
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = __builtin_fmaf(acc_lds[at][c], f, acc[c]);
  }
  const float vscale = p.v_scale != nullptr ? p.v_scale[head / p.group] : 1.f;
  const float f = sum == 0.f ? 0.f : vscale / sum;
  uint16_t* dst = p.out + (int64_t)b * p.ldo + (int64_t)head * p.d + e;
  *reinterpret_cast<u32x2*>(dst) =
      u32x2{(uint32_t)A::round(acc[0] * f) | ((uint32_t)A::round(acc[1] * f) << 16),
            (uint32_t)A::round(acc[2] * f) | ((uint32_t)A::round(acc[3] * f) << 16)};
  if (e == 0 && p.lse != nullptr)
    p.lse[h] = sum == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

// The arguments that every kind of cache has, from the call's (wq_attn_args or wq_attn4_args).  group:
// query heads that count as a KV head's.
template <class Args>
AttnArgs attn_args(const Args& a, const AttnPlan& plan, int group) {
  AttnArgs p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.k = static_cast<const uint8_t*>(a.cache.k);
  p.v = static_cast<const uint8_t*>(a.cache.v);
  p.k_scale = a.cache.k_scale;
  p.v_scale = a.cache.v_scale;
  p.table = a.block_table;
  p.lens = a.lens;
  p.keep = a.keep;
  p.page_stride = a.cache.page_stride;
  p.slot_stride = a.cache.slot_stride;
  p.head_stride = a.cache.head_stride;
  p.num_pages = a.cache.num_pages;
  p.page_size = a.cache.page_size;
  p.kv_heads = a.cache.kv_heads;
  p.q_heads = a.q_heads;
  p.d = a.cache.head_dim;
  p.group = group;
  p.head_blocks = plan.head_blocks;
  p.max_len = a.max_len;
  p.table_stride = a.table_stride;
  p.keep_stride = a.keep_stride;
  p.ldq = a.ldq;
  p.ldo = a.ldo;
  p.window = a.window;
  p.batch = a.batch;
  p.units = plan.units;
  p.part_rows = std::min(p.group, 1 << plan.block_shift);
  p.ranges = plan.ranges;
  p.scale = a.scale;
  p.softcap = a.softcap;
  // exact for positions below 2^30: the multiplier is 2^(31 + shift) / page_size rounded up,
  // with page_size <= 2^shift
  while ((1ll << p.page_shift) < p.page_size) ++p.page_shift;
  p.page_mul = (uint32_t)(((1ull << (31 + p.page_shift)) + p.page_size - 1) / p.page_size);
  if (plan.ranges > 0) {
    const size_t rows = 2 * (size_t)plan.ranges * plan.units * p.part_rows;
    p.part_o = static_cast<float*>(a.workspace);
    p.part_ml = p.part_o + rows * p.d;
    p.parts = reinterpret_cast<int32_t*>(p.part_ml + rows * 2);
  }
  return p;
}

// Work-groups of a launch: a row for each range, or each sequence where there are none.
inline dim3 attn_grid(const AttnArgs& p) {
  size_t rows = p.ranges > 0 ? p.ranges : p.batch;
  if (p.near_units) rows = (rows + 7) / 8 * 8;
  return dim3((unsigned)(rows * p.units));
}

// The second kernel of a call whose sequences are cut.  SHIFT: the plan's block_shift.
template <int SHIFT>
hipError_t launch_attn_join(const AttnArgs& p, bool bf16, hipStream_t stream) {
  const dim3 join((unsigned)p.q_heads, (unsigned)p.batch);
  if (bf16)
    hipLaunchKernelGGL((attn_join_kernel<true, SHIFT>), join, dim3(kJoinThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((attn_join_kernel<false, SHIFT>), join, dim3(kJoinThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace
}  // namespace wq
