// Attention of one new token per sequence over a paged KV cache (wq_paged_attention).
//
// Each live K and V element is read once and takes part in 2 * (query heads per KV head)
// products, so the kernel is bound by the cache reads.  A work-group handles one sequence, one KV head and up to 16
// of its query heads over a range of positions (a split); its waves take tiles of 32
// positions in turn and keep their own running maximum, sum and output, joined at the end
// through LDS.  Splits of long sequences leave fp32 partials that attn_join_kernel adds in
// split order.
//
// Both products run on 16x16x32 MFMAs with the positions as rows:
//  - S^T = K Q^T: the A operand is K straight from memory (a lane holds 8 consecutive
//    elements of one position), the B operand Q.  Lane (row = lane & 15, qd = lane >> 4)
//    then holds the scores of query head `row` at positions 4 qd + e of each 16-position
//    block, so that a head's softmax statistics live in four lanes.
//  - O^T = V^T P^T: the scores' registers are the B operand as they stand, with the sum over
//    positions taken in the order {4 qd + e, 16 + 4 qd + e}; the A operand needs V with
//    positions along the register, which the transposing LDS read gives (16 lanes read a
//    4 x 16 block and each receives a column).  O^T keeps the query head on the lane, so
//    rescaling by the new maximum needs no exchange.
// p = exp(s - max) is split into two 16-bit values, high + low, each in a product of its
// own: the matrix unit has time to spare here, and p keeps at least 16 bits instead of being
// rounded to the element type.  fp16 ends at 2^-24, so there p is formed 2^15 times as large:
// a million positions at 2^-26 of the maximum still count.
//
// One register set serves the loads: K of the next tile is requested when this tile's scores
// are formed, V when this tile's V has gone to LDS, so each wave keeps about a tile in
// flight.  Page numbers are read a tile further ahead.
#include "wq_decode.h"
#include "wq_device.h"

namespace wq {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;  // positions of a wave's step
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Binary places p is raised by (its maximum is 2^kPShift).
template <bool BF16>
constexpr float kPShift = BF16 ? 0.f : 15.f;

struct AttnArgs {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  const int32_t *table, *lens;
  const uint8_t* keep;
  float* part_o;   // [batch][q_heads][splits][d], not divided by the sum
  float* part_ml;  // [batch][q_heads][splits][2]: maximum (times log2 e) and sum
  int64_t page_stride, slot_stride, head_stride;
  int num_pages, page_size, kv_heads, q_heads, d, group, head_blocks, max_len;
  int table_stride, keep_stride, ldq, ldo, window, splits, chunk;
  float scale, softcap;
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Orders a wave's own LDS accesses (they execute in order; this keeps the compiler to it).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <bool BF16>
__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return Act<BF16>::mfma16(a, __builtin_bit_cast(typename Act<BF16>::W8, b), c);
}

template <bool BF16>
__device__ __forceinline__ f16x8 from_e4m3(uint32_t lo, uint32_t hi) {
  return __builtin_bit_cast(f16x8, Act<BF16>::fp8(lo, hi));
}

// DP: head_dim rounded up to 64, 128 or 256.
template <bool BF16, bool KV8, int DP>
__global__ __launch_bounds__(kWaves * 64) void attn_kernel(AttnArgs p) {
  using A = Act<BF16>;
  constexpr int NS = DP / 32;            // MFMA steps along the head
  constexpr int NK = KV8 ? NS / 2 : NS;  // 16-byte K vectors per lane and position block
  constexpr int CE = KV8 ? 16 : 8;       // elements of a 16-byte vector
  constexpr int CPR = DP / CE;           // vectors of a V row
  constexpr int RPI = 64 / CPR;          // V rows of one load
  constexpr int NV = kTile / RPI;
  constexpr int NB = DP / 16;            // 16-element blocks of the output
  constexpr int VS = DP + 16;            // LDS row of V: rows start 8 banks apart
  constexpr int OS = DP + 4;             // LDS row of the joined outputs
  constexpr int kVBytes = kWaves * kTile * VS * 2, kOBytes = kWaves * 16 * OS * 4;
  __shared__ __align__(16) uint8_t lds[kVBytes > kOBytes ? kVBytes : kOBytes];
  __shared__ int64_t off_lds[kWaves][kTile];
  __shared__ float ml_lds[kWaves][16][2];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, qd = lane >> 4;
  const int split = blockIdx.x, b = blockIdx.z;
  const int kvh = blockIdx.y / p.head_blocks, hb = blockIdx.y - kvh * p.head_blocks;
  const int h0 = kvh * p.group + 16 * hb;         // first query head
  const int rows = min(16, p.group - 16 * hb);
  const int len = max(0, min(p.lens[b], p.max_len));
  const int lo = p.window > 0 ? max(0, len - p.window) : 0;  // first live position
  const int t0 = (lo & ~(kTile - 1)) + split * p.chunk;
  const int t1 = min(len, t0 + p.chunk);
  if (t0 >= t1) {  // nothing in this split
    for (int i = threadIdx.x; i < rows; i += kWaves * 64) {
      const int64_t h = (int64_t)b * p.q_heads + h0 + i;
      if (p.splits > 1) {
        p.part_ml[(h * p.splits + split) * 2] = -INFINITY;
        p.part_ml[(h * p.splits + split) * 2 + 1] = 0.f;
      } else if (p.lse != nullptr) {
        p.lse[h] = -INFINITY;
      }
    }
    if (p.splits == 1)
      for (int i = threadIdx.x; i < rows * p.d; i += kWaves * 64)
        p.out[(int64_t)b * p.ldo + (int64_t)h0 * p.d + i] = 0;
    return;
  }

  // Q as the B operand; query heads past the last repeat the first (never stored).
  f16x8 qf[NS];
  {
    const uint16_t* qp = p.q + (int64_t)b * p.ldq + (int64_t)(h0 + (row < rows ? row : 0)) * p.d;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int e = KV8 ? 64 * (s / 2) + 16 * qd + 8 * (s % 2) : 32 * s + 8 * qd;
      qf[s] = f16x8{};
      if (e < p.d) qf[s] = *reinterpret_cast<const f16x8*>(qp + e);
    }
  }

  const uint8_t* kbase = p.k + kvh * p.head_stride * (KV8 ? 1 : 2);
  const uint8_t* vbase = p.v + kvh * p.head_stride * (KV8 ? 1 : 2);
  const int32_t* table = p.table + (int64_t)b * p.table_stride;
  const uint8_t* keep = p.keep != nullptr ? p.keep + (int64_t)b * p.keep_stride : nullptr;

  // A vector that lies past the head's end is read from its start and not used; an E4M3
  // vector that passes the end half way (head_dim % 16 == 8) is read 8 bytes earlier and
  // shifted.
  const auto vec_at = [&](int e) { return e + CE <= p.d ? e : (e < p.d ? p.d - CE : 0); };
  const auto vec_fix = [&](u32x4 w, int e) {
    if (KV8 && e < p.d && e + CE > p.d) w = u32x4{w[2], w[3], 0u, 0u};
    return e < p.d ? w : u32x4{0u, 0u, 0u, 0u};
  };

  // Page numbers (and keep bytes) of the tile at t, one position per lane and half-wave.
  int page_next = -1;
  const auto read_pages = [&](int t) {
    const int pos = t + (lane & (kTile - 1));
    page_next = -1;
    if (pos >= lo && pos < t1) {
      page_next = table[pos / p.page_size];
      if (keep != nullptr && keep[pos] == 0) page_next = -1;
    }
  };
  // Cache offsets of the tile at t, from page_next; returns the mask of live positions.  A
  // position that is not live reads the cache's first slot, and is not used.
  const auto place = [&](int t) -> uint32_t {
    const int pos = t + (lane & (kTile - 1));
    const bool live = (unsigned)page_next < (unsigned)p.num_pages;
    const int slot = pos - pos / p.page_size * p.page_size;
    off_lds[wave][lane & (kTile - 1)] =
        live ? page_next * p.page_stride + slot * p.slot_stride : 0;
    return (uint32_t)__ballot(live);
  };
  u32x4 kr[2][NK], vr[NV];
  const auto load_k = [&] {
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      const uint8_t* kp = kbase + off_lds[wave][16 * blk + row] * (KV8 ? 1 : 2);
#pragma unroll
      for (int s = 0; s < NK; ++s)
        kr[blk][s] = *reinterpret_cast<const u32x4*>(
            kp + vec_at(4 * CE * s + CE * qd) * (KV8 ? 1 : 2));
    }
  };
  const int vcol = CE * (lane % CPR);
  const auto load_v = [&] {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      vr[j] = *reinterpret_cast<const u32x4*>(
          vbase + (off_lds[wave][j * RPI + lane / CPR] + vec_at(vcol)) * (KV8 ? 1 : 2));
  };

  uint16_t* const v_lds = reinterpret_cast<uint16_t*>(lds) + wave * kTile * VS;
  const float kscale = KV8 && p.k_scale != nullptr ? p.k_scale[kvh] : 1.f;
  const float sc = p.scale * kscale;
  float m = -INFINITY, l = 0.f;
  f32x4 o[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};

  constexpr int kStep = kWaves * kTile;
  int t = t0 + wave * kTile;
  uint32_t live = 0;
  if (t < t1) {
    read_pages(t);
    wave_lds_fence();
    live = place(t);
    wave_lds_fence();
    read_pages(t + kStep);
    load_k();
    load_v();
  }
  for (; t < t1; t += kStep) {
    // scores
    f32x4 s[2];
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      s[blk] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        f16x8 kf;
        if constexpr (KV8) {
          const u32x4 w = vec_fix(kr[blk][i / 2], 64 * (i / 2) + 16 * qd);
          kf = from_e4m3<BF16>(w[2 * (i % 2)], w[2 * (i % 2) + 1]);
        } else {
          kf = __builtin_bit_cast(f16x8, vec_fix(kr[blk][i], 32 * i + 8 * qd));
        }
        s[blk] = mfma<BF16>(kf, qf[i], s[blk]);
      }
    }
    const uint32_t now = live;
    // the next tile's K (positions past the range are not live and read the first slot)
    wave_lds_fence();
    live = place(t + kStep);
    wave_lds_fence();
    read_pages(t + 2 * kStep);
    load_k();

    // running maximum and sum, in base 2
    float mx = -INFINITY;
#pragma unroll
    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = s[blk][e] * sc;
        if (p.softcap > 0.f) x = p.softcap * tanhf(x / p.softcap);
        x *= kLog2e;
        x = (now >> (16 * blk + 4 * qd + e)) & 1u ? x : -INFINITY;
        s[blk][e] = x;
        mx = fmaxf(mx, x);
      }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float m_new = fmaxf(m, mx);
    const float top = m_new == -INFINITY ? 0.f : m_new;  // nothing live so far
    const float ref = top - kPShift<BF16>;
    const float alpha = __builtin_amdgcn_exp2f(m - top);
    m = m_new;
    l *= alpha;
    uint16_t hi[8], lw[8];
#pragma unroll
    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = __builtin_amdgcn_exp2f(s[blk][e] - ref);
        l += x;
        const uint16_t h = A::round(x);
        hi[4 * blk + e] = h;
        lw[4 * blk + e] = A::round(x - A::value(h));
      }
    f16x8 ph, pl;
    __builtin_memcpy(&ph, hi, 16);
    __builtin_memcpy(&pl, lw, 16);

    // V to LDS as 16-bit rows, zero where a position is not live
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int r = j * RPI + lane / CPR;
      u32x4 w = vec_fix(vr[j], vcol);
      if (now != 0xFFFFFFFFu && !((now >> r) & 1u)) w = u32x4{0u, 0u, 0u, 0u};
      if constexpr (KV8) {
        *reinterpret_cast<f16x8*>(v_lds + r * VS + vcol) = from_e4m3<BF16>(w[0], w[1]);
        *reinterpret_cast<f16x8*>(v_lds + r * VS + vcol + 8) = from_e4m3<BF16>(w[2], w[3]);
      } else {
        *reinterpret_cast<u32x4*>(v_lds + r * VS + vcol) = w;
      }
    }
    wave_lds_fence();
    load_v();

#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint16_t* src = v_lds + (4 * qd + (row >> 2)) * VS + 16 * i + 4 * (row & 3);
      const s16x4 a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)src);
      const s16x4 a1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(src + 16 * VS));
      f16x8 vf;
      __builtin_memcpy(&vf, &a0, 8);
      __builtin_memcpy(reinterpret_cast<char*>(&vf) + 8, &a1, 8);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] *= alpha;
      o[i] = mfma<BF16>(vf, ph, o[i]);
      o[i] = mfma<BF16>(vf, pl, o[i]);
    }
    wave_lds_fence();
  }

  // Join the waves, in wave order.
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  __syncthreads();  // every wave is done with its V rows
  float* const o_lds = reinterpret_cast<float*>(lds);
  if (qd == 0) {
    ml_lds[wave][row][0] = m - kPShift<BF16>;
    ml_lds[wave][row][1] = l;
  }
#pragma unroll
  for (int i = 0; i < NB; ++i)
    *reinterpret_cast<f32x4*>(o_lds + (wave * 16 + row) * OS + 16 * i + 4 * qd) = o[i];
  __syncthreads();
  const int per_row = p.d / 4;
  const float vscale = KV8 && p.v_scale != nullptr ? p.v_scale[kvh] : 1.f;
  for (int i = threadIdx.x; i < rows * per_row; i += kWaves * 64) {
    const int r = i / per_row, e = 4 * (i - r * per_row);
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, ml_lds[w][r][0]);
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(ml_lds[w][r][0] - ref);
      sum = __builtin_fmaf(ml_lds[w][r][1], f, sum);
      const f32x4 x = *reinterpret_cast<const f32x4*>(o_lds + (w * 16 + r) * OS + e);
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = __builtin_fmaf(x[c], f, acc[c]);
    }
    const int64_t h = (int64_t)b * p.q_heads + h0 + r;
    if (p.splits > 1) {
      *reinterpret_cast<f32x4*>(p.part_o + (h * p.splits + split) * p.d + e) = acc;
      if (e == 0) {
        p.part_ml[(h * p.splits + split) * 2] = top;
        p.part_ml[(h * p.splits + split) * 2 + 1] = sum;
      }
    } else {
      const float f = sum == 0.f ? 0.f : vscale / sum;
      uint16_t* dst = p.out + (int64_t)b * p.ldo + (int64_t)(h0 + r) * p.d + e;
      *reinterpret_cast<u32x2*>(dst) =
          u32x2{(uint32_t)A::round(acc[0] * f) | ((uint32_t)A::round(acc[1] * f) << 16),
                (uint32_t)A::round(acc[2] * f) | ((uint32_t)A::round(acc[3] * f) << 16)};
      if (e == 0 && p.lse != nullptr)
        p.lse[h] = sum == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
    }
  }
}

// Joins the splits of one query head: groups of threads, each d / 4 wide, take splits in
// turn and are added in group order.
constexpr int kJoinThreads = 256;

template <bool BF16>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs p) {
  using A = Act<BF16>;
  __shared__ f32x4 acc_lds[kJoinThreads];
  __shared__ float sum_lds[kJoinThreads];
  const int head = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int64_t h = (int64_t)b * p.q_heads + head;
  const int per_row = p.d / 4;  // at most 64
  const int groups = kJoinThreads / per_row;
  const int g = tid / per_row, e = 4 * (tid - g * per_row);
  const float* ml = p.part_ml + h * p.splits * 2;
  const float* po = p.part_o + h * p.splits * p.d;

  float top = -INFINITY;
  for (int s = tid; s < p.splits; s += kJoinThreads) top = fmaxf(top, ml[2 * s]);
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) top = fmaxf(top, __shfl_xor(top, d));
  if ((tid & 63) == 0) sum_lds[tid >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(sum_lds[0], sum_lds[1]), fmaxf(sum_lds[2], sum_lds[3]));
  __syncthreads();
  const float ref = top == -INFINITY ? 0.f : top;

  float sum = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (g < groups) {
    for (int s = g; s < p.splits; s += groups) {
      const float ms = ml[2 * s], ls = ml[2 * s + 1];
      if (ms == -INFINITY && ls == 0.f) continue;  // an empty split wrote no sums
      const float f = __builtin_amdgcn_exp2f(ms - ref);
      sum = __builtin_fmaf(ls, f, sum);
      const f32x4 x = *reinterpret_cast<const f32x4*>(po + (int64_t)s * p.d + e);
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = __builtin_fmaf(x[c], f, acc[c]);
    }
  }
  acc_lds[tid] = acc;
  sum_lds[tid] = sum;
  __syncthreads();
  if (g != 0) return;
  for (int k = 1; k < groups; ++k) {
    sum += sum_lds[tid + k * per_row];
    acc += acc_lds[tid + k * per_row];
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

}  // namespace

AttnPlan attn_plan(int batch, int q_heads, int kv_heads, int head_dim, int max_len, int window) {
  AttnPlan plan{};
  plan.head_blocks = (q_heads / kv_heads + 15) / 16;
  // positions a sequence may need, from the tile that holds the window's first
  const long span = window > 0 && window < max_len - kTile ? window + kTile - 1 : max_len;
  const long units = (long)batch * kv_heads * plan.head_blocks;
  constexpr long kStep = kWaves * kTile;
  long chunk = span * units / 1024;
  if (chunk < 2 * kStep) chunk = 2 * kStep;
  chunk = (chunk + kStep - 1) / kStep * kStep;
  (void)head_dim;
  plan.chunk = (int)chunk;
  plan.splits = (int)((span + chunk - 1) / chunk);
  return plan;
}

size_t attn_workspace_bytes(const AttnPlan& plan, int batch, int q_heads, int head_dim) {
  if (plan.splits <= 1) return 0;
  return (size_t)batch * q_heads * plan.splits * (head_dim + 2) * sizeof(float);
}

hipError_t launch_paged_attention(const wq_attn_args& a, const AttnPlan& plan,
                                  hipStream_t stream) {
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
  p.group = a.q_heads / a.cache.kv_heads;
  p.head_blocks = plan.head_blocks;
  p.max_len = a.max_len;
  p.table_stride = a.table_stride;
  p.keep_stride = a.keep_stride;
  p.ldq = a.ldq;
  p.ldo = a.ldo;
  p.window = a.window;
  p.splits = plan.splits;
  p.chunk = plan.chunk;
  p.scale = a.scale;
  p.softcap = a.softcap;
  if (plan.splits > 1) {
    p.part_o = static_cast<float*>(a.workspace);
    p.part_ml = p.part_o + (size_t)a.batch * a.q_heads * plan.splits * p.d;
  }
  const bool bf16 = (a.flags & WQ_FLAG_BF16) != 0, kv8 = (a.flags & WQ_FLAG_FP8) != 0;
  const dim3 grid((unsigned)plan.splits, (unsigned)(p.kv_heads * plan.head_blocks),
                  (unsigned)a.batch);
#define WQ_ATTN(B, F, D)                                                                      \
  hipLaunchKernelGGL((attn_kernel<B, F, D>), grid, dim3(kWaves * 64), 0, stream, p)
#define WQ_ATTN_D(B, F)                                                                       \
  do {                                                                                        \
    if (p.d <= 64) WQ_ATTN(B, F, 64);                                                         \
    else if (p.d <= 128) WQ_ATTN(B, F, 128);                                                  \
    else WQ_ATTN(B, F, 256);                                                                  \
  } while (0)
  if (bf16) {
    if (kv8) WQ_ATTN_D(true, true); else WQ_ATTN_D(true, false);
  } else {
    if (kv8) WQ_ATTN_D(false, true); else WQ_ATTN_D(false, false);
  }
#undef WQ_ATTN_D
#undef WQ_ATTN
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.splits == 1) return e;
  const dim3 join((unsigned)a.q_heads, (unsigned)a.batch);
  if (bf16)
    hipLaunchKernelGGL((attn_join_kernel<true>), join, dim3(kJoinThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((attn_join_kernel<false>), join, dim3(kJoinThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace wq
