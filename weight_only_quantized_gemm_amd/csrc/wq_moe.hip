// A whole mixture-of-experts layer of a few tokens (wq_moe_layer): routing, the chosen
// experts' gate/up projections with SwiGLU, their down projections and the weighted sum.
//
// The layer reads every chosen expert's weights once and does 2 * (rows per expert) products
// per weight, so it is bound by the weight stream.  Four kernels, each needing the whole
// result of the one before it:
//  1. router_kernel: the logits x router^T.
//  2. route_kernel (one work-group): top-k and weights per token, then the experts that were
//     chosen at all ("slots"), which tokens each has, and where its rows of the activation
//     buffer start.  Nothing returns to the host: the next grids are sized for the most slots
//     there can be, and work-groups past the last slot end at once.
//  3. gate_up_kernel: one work-group per pair of 16-column blocks and slot.
//  4. down_kernel: one work-group per 16 output columns walks all slots, so the weighted sum
//     over a token's experts is formed in registers, in a fixed order, and no pair rows or
//     atomics are needed.
// Products are 16x16x32 MFMAs on codes dequantized in registers (wq_device.h); each scale
// unit's partial is scaled in fp32.
#include "wq_decode.h"
#include "wq_device.h"

namespace wq {
namespace {

constexpr int kMaxT = WQ_MOE_MAX_TOKENS;
constexpr int kMaxE = WQ_MOE_MAX_EXPERTS;

// The routing of a call, in the workspace.
struct Route {
  int32_t n_active;
  int32_t pad[3];
  int32_t expert[kMaxE];   // of each slot, ascending
  uint32_t mask[kMaxE];    // its tokens
  int32_t off[kMaxE];      // its first row of the activation buffer
  float w[kMaxE][kMaxT];   // routing weight of each token (0 where not routed)
};

struct Bank {
  const u32x4* b;
  const uint16_t* s;
  const u32x2* z;
  long b_stride, s_stride, z_stride;  // in elements of the above
};

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// ---- routing ---------------------------------------------------------------------------

// Logits of one expert and four tokens per wave.  Eight products at a time are summed in
// fp32, the sums in fp64: the order of nearly equal logits decides which experts run.
template <bool BF16>
__global__ __launch_bounds__(256) void router_kernel(const uint16_t* __restrict__ x, int ldx,
                                                     const uint16_t* __restrict__ router,
                                                     int tokens, int n_expert, int hidden,
                                                     double* __restrict__ logits) {
  using A = Act<BF16>;
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int t0 = blockIdx.y * 4;
  if (e >= n_expert) return;
  const uint16_t* rp = router + (long)e * hidden;
  double acc[4] = {0., 0., 0., 0.};
#pragma unroll 2
  for (int k = lane * 8; k < hidden; k += 512) {
    const u32x4 r = *reinterpret_cast<const u32x4*>(rp + k);
    float rf[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rf[i] = A::value((uint16_t)(r[i / 2] >> (16 * (i % 2))));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + j < tokens ? t0 + j : tokens - 1;
      const u32x4 xv = *reinterpret_cast<const u32x4*>(x + (long)t * ldx + k);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        sum = __builtin_fmaf(rf[i], A::value((uint16_t)(xv[i / 2] >> (16 * (i % 2)))), sum);
      acc[j] += (double)sum;
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d /= 2)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], d);
  if (lane < 4 && t0 + lane < tokens) {
    double v = acc[0];
#pragma unroll
    for (int j = 1; j < 4; ++j) v = lane == j ? acc[j] : v;
    logits[(t0 + lane) * n_expert + e] = v;
  }
}

template <int CTRL>
__device__ __forceinline__ double dpp_max(double x) {
  const long long bits = __builtin_bit_cast(long long, x);
  const int lo = __builtin_amdgcn_update_dpp((int)bits, (int)bits, CTRL, 0xf, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp((int)(bits >> 32), (int)(bits >> 32), CTRL, 0xf,
                                             0xf, false);
  const double other =
      __builtin_bit_cast(double, ((long long)hi << 32) | (long long)(unsigned)lo);
  return other > x ? other : x;
}

// Maximum over the wave, in every lane.
__device__ __forceinline__ double wave_max(double x) {
  x = dpp_max<0x111>(x);  // row_shr 1, 2, 4, 8: lane 15 of each row of 16 has its maximum
  x = dpp_max<0x112>(x);
  x = dpp_max<0x114>(x);
  x = dpp_max<0x118>(x);
  x = dpp_max<0x142>(x);  // row_bcast 15 and 31: lane 63 has the wave's
  x = dpp_max<0x143>(x);
  const long long bits = __builtin_bit_cast(long long, x);
  const unsigned lo = __builtin_amdgcn_readlane((int)bits, 63);
  const int hi = __builtin_amdgcn_readlane((int)(bits >> 32), 63);
  return __builtin_bit_cast(double, ((long long)hi << 32) | (long long)lo);
}

// Wave t takes token t's top-k.  Each logit's lowest 8 mantissa bits give way to its expert
// number, coded so that of equal logits the lower expert is the larger key.
__global__ __launch_bounds__(kMaxT * 64) void route_kernel(const double* __restrict__ logits,
                                                          int tokens, int n_expert, int top_k,
                                                          int renormalize, float routed_scale,
                                                          int32_t* __restrict__ ids,
                                                          float* __restrict__ weights,
                                                          Route* __restrict__ route) {
  constexpr int PER = kMaxE / 64;
  __shared__ uint32_t mask_lds[kMaxE];
  __shared__ float w_lds[kMaxE][kMaxT];
  __shared__ int total_lds[PER][2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int t = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int i = tid; i < kMaxE; i += kMaxT * 64) mask_lds[i] = 0;
  for (int i = tid; i < n_expert * kMaxT; i += kMaxT * 64) w_lds[i / kMaxT][i % kMaxT] = 0.f;
  __syncthreads();
  if (t < tokens) {
    double l[PER], key[PER];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 64 * i;
      l[i] = e < n_expert ? logits[t * n_expert + e] : -INFINITY;
      bad |= l[i] != l[i] || l[i] == INFINITY;
      const double big = 1e300;
      double c = l[i] > -big ? (l[i] < big ? l[i] : big) : -big;  // NaN: lowest
      if (l[i] == INFINITY) c = big;
      c += 0.0;  // -0 and 0 are equal
      unsigned long long bits = __builtin_bit_cast(unsigned long long, c);
      bits = (bits & ~255ull) | (unsigned long long)((bits >> 63) ? e : 255 - e);
      key[i] = e < n_expert ? __builtin_bit_cast(double, bits) : -INFINITY;
    }
    const bool nan_row = __ballot(bad) != 0;
    double top = 0.;
    float chosen = 0.f, mine = 0.f;
    int my_id = 0;
    for (int j = 0; j < top_k; ++j) {
      double best = key[0];
#pragma unroll
      for (int i = 1; i < PER; ++i) best = key[i] > best ? key[i] : best;
      best = wave_max(best);
      if (j == 0) top = best;
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = key[i] == best ? -INFINITY : key[i];
      const unsigned long long bits = __builtin_bit_cast(unsigned long long, best);
      const int code = (int)(bits & 255ull);
      const float w = expf((float)(best - top));
      chosen += w;
      if (lane == j) {
        mine = w;
        my_id = (bits >> 63) ? code : 255 - code;
      }
    }
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) all += expf((float)(l[i] - top));
#pragma unroll
    for (int d = 32; d >= 1; d /= 2) all += __shfl_xor(all, d);
    const float sum = renormalize ? chosen : all;
    // a row without a finite logit has no softmax
    float w = nan_row || !(all > 0.f) ? __builtin_nanf("") : mine / sum;
    if (lane < top_k) {
      if (ids != nullptr) ids[t * top_k + lane] = my_id;
      w *= routed_scale;
      if (weights != nullptr) weights[t * top_k + lane] = w;
      w_lds[my_id][t] = w;
      atomicOr(&mask_lds[my_id], 1u << t);
    }
  }
  __syncthreads();
  // Thread e of the first waves: expert e's slot and first row, counted over lower experts.
  uint32_t m = 0;
  int slot = 0, off = 0;
  if (tid < kMaxE) {
    m = mask_lds[tid];
    const unsigned long long below = (1ull << lane) - 1;
    const unsigned long long act = __ballot(m != 0);
    slot = __popcll(act & below);
    int rows = 0;
#pragma unroll
    for (int i = 0; i < kMaxT; ++i) {
      const unsigned long long has = __ballot((m >> i) & 1u);
      off += __popcll(has & below);
      rows += __popcll(has);
    }
    if (lane == 0) {
      total_lds[t][0] = __popcll(act);
      total_lds[t][1] = rows;
    }
  }
  __syncthreads();
  if (tid < kMaxE) {
    int active = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (i < t) {
        slot += total_lds[i][0];
        off += total_lds[i][1];
      }
      active += total_lds[i][0];
    }
    if (tid == 0) route->n_active = active;
    if (m != 0) {
      route->expert[slot] = tid;
      route->mask[slot] = m;
      route->off[slot] = off;
#pragma unroll
      for (int i = 0; i < kMaxT; i += 4)
        *reinterpret_cast<f32x4*>(&route->w[slot][i]) =
            *reinterpret_cast<const f32x4*>(&w_lds[tid][i]);
    }
  }
}

// ---- the quantized products ------------------------------------------------------------

// One 128-row chunk of a 16-column block as its wave holds it: codes, scales, zero points.
template <bool BF16, bool W8, bool ZP, int GPC>
struct Chunk {
  using A = Act<BF16>;
  u32x4 w[W8 ? 2 : 1];
  uint16_t s[GPC];
  u32x2 z[ZP ? GPC : 1];

  // at: chunk index of the expert's layout (block * groups + group)
  __device__ __forceinline__ void load(const u32x4* b, const uint16_t* sp, const u32x2* zp,
                                       long at, int lane) {
#pragma unroll
    for (int v = 0; v < (W8 ? 2 : 1); ++v)
      w[v] = __builtin_nontemporal_load(b + (at * (W8 ? 2 : 1) + v) * 64 + lane);
#pragma unroll
    for (int u = 0; u < GPC; ++u) s[u] = sp[(at * GPC + u) * 16 + (lane & 15)];
    if constexpr (ZP) {
#pragma unroll
      for (int u = 0; u < GPC; ++u) z[u] = zp[at * GPC + u];
    }
  }

  // acc += (16 rows of A, four 32-row steps) x chunk
  __device__ __forceinline__ void multiply(const f16x8* a, int lane, f32x4& acc) const {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const auto add = [&](uint16_t scale, f32x4 part) {
      const float f = A::value(scale);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(f, part[e], acc[e]);
    };
    const auto offsets = [&](int u) { return A::zero(ZP ? zero_code(z[ZP ? u : 0], lane & 15) : 8); };
    if constexpr (W8) {
      f32x4 p = zero;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        p = A::mfma16(a[j], A::fp8(w[j / 2][2 * (j % 2)], w[j / 2][2 * (j % 2) + 1]), p);
      add(s[0], p);
    } else if constexpr (GPC <= 4) {
      const auto mr = A::magic();
      constexpr int JQ = 4 / GPC;
#pragma unroll
      for (int u = 0; u < GPC; ++u) {
        const auto zo = offsets(u);
        f32x4 p = zero;
#pragma unroll
        for (int j = JQ * u; j < JQ * (u + 1); ++j)
          p = A::mfma16(a[j], A::dequant(w[0][j], zo, mr), p);
        add(s[u], p);
      }
    } else {
      // 16-row units: lanes 0-31 hold a step's first unit, lanes 32-63 its second; each unit
      // has its product, the other half's weights set to zero
      const auto mr = A::magic();
      const bool second = lane >= 32;
      const typename A::W8 none{};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const auto z0 = offsets(2 * j), z1 = offsets(2 * j + 1);
        const typename A::W8 q = second ? A::dequant(w[0][j], z1, mr) : A::dequant(w[0][j], z0, mr);
        add(s[2 * j], A::mfma16(a[j], second ? none : q, zero));
        add(s[2 * j + 1], A::mfma16(a[j], second ? q : none, zero));
      }
    }
  }
};

__device__ __forceinline__ void load_rows(const uint16_t* row_at, int g, f16x8* a) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    a[j] = *reinterpret_cast<const f16x8*>(row_at + (long)g * kGroup + 32 * j);
}

constexpr int kGuWaves = 8;
constexpr int kGuUnroll = 2;

template <bool BF16, bool W8, bool ZP, int GPC>
__global__ __launch_bounds__(kGuWaves * 64) void gate_up_kernel(
    const uint16_t* __restrict__ x, int ldx, Bank bank, const Route* __restrict__ route,
    int groups, int inter, uint16_t* __restrict__ h) {
  using A = Act<BF16>;
  using C = Chunk<BF16, W8, ZP, GPC>;
  __shared__ f32x4 red[2][kGuWaves][64];
  const int slot = blockIdx.y;
  if (slot >= route->n_active) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long expert = route->expert[slot];
  const uint32_t mask = route->mask[slot];
  const int off = route->off[slot];
  const int rows = __popc(mask);
  const u32x4* b = bank.b + expert * bank.b_stride;
  const uint16_t* s = bank.s + expert * bank.s_stride;
  const u32x2* z = ZP ? bank.z + expert * bank.z_stride : nullptr;

  // Row r of the block is the slot's r-th token; rows past the last repeat the first.
  uint32_t rest = mask;
  for (int i = 0; i < (lane & 15) && (lane & 15) < rows; ++i) rest &= rest - 1;
  const int token = __ffs(rest) - 1;
  const uint16_t* xp = x + (long)token * ldx + 8 * (lane >> 4);

  const long gate0 = 2L * blockIdx.x * groups, up0 = gate0 + groups;
  f32x4 gate = {0.f, 0.f, 0.f, 0.f}, up = gate;
  for (int g0 = wave; g0 < groups; g0 += kGuWaves * kGuUnroll) {
    C cg[kGuUnroll], cu[kGuUnroll];
    f16x8 a[kGuUnroll][4];
#pragma unroll
    for (int i = 0; i < kGuUnroll; ++i) {
      const int g = min(g0 + i * kGuWaves, groups - 1);
      cg[i].load(b, s, z, gate0 + g, lane);
      cu[i].load(b, s, z, up0 + g, lane);
      load_rows(xp, g, a[i]);
    }
#pragma unroll
    for (int i = 0; i < kGuUnroll; ++i) {
      if (g0 + i * kGuWaves >= groups) continue;
      cg[i].multiply(a[i], lane, gate);
      cu[i].multiply(a[i], lane, up);
    }
  }
  red[0][wave][lane] = gate;
  red[1][wave][lane] = up;
  __syncthreads();
  if (wave >= 4) return;
  // wave e sums element e of the lane's block, in wave order
  const int e = wave, r = 4 * (lane >> 4) + e;
  float gs = 0.f, us = 0.f;
#pragma unroll
  for (int w = 0; w < kGuWaves; ++w) {
    gs += reinterpret_cast<const float*>(&red[0][w][lane])[e];
    us += reinterpret_cast<const float*>(&red[1][w][lane])[e];
  }
  if (r < rows) h[(long)(off + r) * inter + 16 * blockIdx.x + (lane & 15)] = A::round(silu_times(gs, us));
}

constexpr int kDnWaves = 16;
constexpr int kDnUnroll = 4;

template <bool BF16, bool W8, bool ZP, int GPC>
__global__ __launch_bounds__(kDnWaves * 64) void down_kernel(
    const uint16_t* __restrict__ h, Bank bank, const Route* __restrict__ route, int groups,
    int inter, const uint16_t* residual, int ldr, uint16_t* y, int ldy, int tokens) {
  using A = Act<BF16>;
  using C = Chunk<BF16, W8, ZP, GPC>;
  __shared__ f32x4 red[kDnWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, qd = lane >> 4;
  const long block0 = (long)blockIdx.x * groups;

  // (slot, group) items in slot order; each wave takes a run of them
  const int items = route->n_active * groups;
  int i = (int)((long)items * wave / kDnWaves);
  const int last = (int)((long)items * (wave + 1) / kDnWaves);
  f32x4 total = {0.f, 0.f, 0.f, 0.f};
  while (i < last) {
    const int slot = i / groups;
    const int g1 = min(last - slot * groups, groups);
    const long expert = route->expert[slot];
    const uint32_t mask = route->mask[slot];
    const f32x4 w = *reinterpret_cast<const f32x4*>(&route->w[slot][4 * qd]);
    const u32x4* b = bank.b + expert * bank.b_stride;
    const uint16_t* s = bank.s + expert * bank.s_stride;
    const u32x2* z = ZP ? bank.z + expert * bank.z_stride : nullptr;
    // Row t of the block is token t; a token without this expert reads the slot's first row
    // (its sums are left out below).
    const int r = (mask >> row) & 1u ? __popc(mask & ((1u << row) - 1)) : 0;
    const uint16_t* hp = h + (long)(route->off[slot] + r) * inter + 8 * qd;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int g0 = i - slot * groups; g0 < g1; g0 += kDnUnroll) {
      C c[kDnUnroll];
      f16x8 a[kDnUnroll][4];
#pragma unroll
      for (int k = 0; k < kDnUnroll; ++k) {
        const int g = min(g0 + k, g1 - 1);
        c[k].load(b, s, z, block0 + g, lane);
        load_rows(hp, g, a[k]);
      }
#pragma unroll
      for (int k = 0; k < kDnUnroll; ++k)
        if (g0 + k < g1) c[k].multiply(a[k], lane, acc);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      total[e] = (mask >> (4 * qd + e)) & 1u ? __builtin_fmaf(w[e], acc[e], total[e]) : total[e];
    i = slot * groups + g1;
  }
  red[wave][lane] = total;
  __syncthreads();
  if (wave >= 4) return;
  const int e = wave, t = 4 * qd + e;
  if (t >= tokens) return;
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < kDnWaves; ++k) sum += reinterpret_cast<const float*>(&red[k][lane])[e];
  const long col = 16L * blockIdx.x + row;
  if (residual != nullptr) sum += A::value(residual[(long)t * ldr + col]);
  y[(long)t * ldy + col] = A::round(sum);
}

int max_slots(int tokens, int n_expert, int top_k) {
  return tokens * top_k < n_expert ? tokens * top_k : n_expert;
}

Bank bank_of(const wq_expert_bank& b) {
  return Bank{static_cast<const u32x4*>(b.b), static_cast<const uint16_t*>(b.s),
              static_cast<const u32x2*>(b.zp), (long)(b.b_stride_bytes / 16),
              (long)(b.s_stride_bytes / 2), (long)(b.zp_stride_bytes / 8)};
}

struct MoeScratch {
  double* logits;
  Route* route;
  uint16_t* h;
  size_t bytes;
};

MoeScratch scratch_of(void* base, int tokens, int n_expert, int top_k, int inter) {
  const size_t logits = round256((size_t)tokens * n_expert * sizeof(double));
  const size_t route = round256(sizeof(Route));
  char* p = static_cast<char*>(base);
  return MoeScratch{reinterpret_cast<double*>(p), reinterpret_cast<Route*>(p + logits),
                    reinterpret_cast<uint16_t*>(p + logits + route),
                    logits + route + round256((size_t)tokens * top_k * inter * 2)};
}

template <bool BF16, bool W8, bool ZP, int GPC>
hipError_t launch_gate_up(const wq_moe_args& a, const MoeScratch& m, hipStream_t stream) {
  const dim3 grid(a.inter / 16, max_slots(a.tokens, a.n_expert, a.top_k));
  hipLaunchKernelGGL((gate_up_kernel<BF16, W8, ZP, GPC>), grid, dim3(kGuWaves * 64), 0, stream,
                     static_cast<const uint16_t*>(a.x), a.ldx, bank_of(a.gate_up), m.route,
                     a.hidden / kGroup, a.inter, m.h);
  return hipGetLastError();
}

template <bool BF16, bool W8, bool ZP, int GPC>
hipError_t launch_down(const wq_moe_args& a, const MoeScratch& m, hipStream_t stream) {
  hipLaunchKernelGGL((down_kernel<BF16, W8, ZP, GPC>), dim3(a.hidden / 16), dim3(kDnWaves * 64),
                     0, stream, m.h, bank_of(a.down), m.route, a.inter / kGroup, a.inter,
                     static_cast<const uint16_t*>(a.residual), a.ldr,
                     static_cast<uint16_t*>(a.y), a.ldy, a.tokens);
  return hipGetLastError();
}

template <bool BF16, bool W8, bool ZP, int GPC>
hipError_t launch_product(bool down, const wq_moe_args& a, const MoeScratch& m,
                          hipStream_t stream) {
  return down ? launch_down<BF16, W8, ZP, GPC>(a, m, stream)
              : launch_gate_up<BF16, W8, ZP, GPC>(a, m, stream);
}

template <bool BF16>
hipError_t launch_product_type(bool down, int gpc, const wq_moe_args& a, const MoeScratch& m,
                               hipStream_t stream) {
  if (a.flags & WQ_FLAG_FP8) return launch_product<BF16, true, false, 1>(down, a, m, stream);
  const bool zp = (a.flags & WQ_FLAG_HAS_ZP) != 0;
  switch (gpc) {
#define WQ_MOE_GPC(G)                                                            \
  case G:                                                                        \
    return zp ? launch_product<BF16, false, true, G>(down, a, m, stream)         \
              : launch_product<BF16, false, false, G>(down, a, m, stream)
    WQ_MOE_GPC(1);
    WQ_MOE_GPC(2);
    WQ_MOE_GPC(4);
    WQ_MOE_GPC(8);
#undef WQ_MOE_GPC
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

size_t moe_workspace_bytes(int tokens, int n_expert, int top_k, int hidden, int inter) {
  (void)hidden;
  return scratch_of(nullptr, tokens, n_expert, top_k, inter).bytes;
}

hipError_t launch_moe_layer(const wq_moe_args& a, int gate_up_gpc, int down_gpc,
                            hipStream_t stream) {
  const MoeScratch m = scratch_of(a.workspace, a.tokens, a.n_expert, a.top_k, a.inter);
  const bool bf16 = (a.flags & WQ_FLAG_BF16) != 0;
  const dim3 grid((a.n_expert + 3) / 4, (a.tokens + 3) / 4);
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  const uint16_t* r = static_cast<const uint16_t*>(a.router);
  if (bf16)
    hipLaunchKernelGGL((router_kernel<true>), grid, dim3(256), 0, stream, x, a.ldx, r, a.tokens,
                       a.n_expert, a.hidden, m.logits);
  else
    hipLaunchKernelGGL((router_kernel<false>), grid, dim3(256), 0, stream, x, a.ldx, r, a.tokens,
                       a.n_expert, a.hidden, m.logits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(route_kernel, dim3(1), dim3(kMaxT * 64), 0, stream, m.logits, a.tokens,
                     a.n_expert, a.top_k, a.renormalize, a.routed_scale, a.ids, a.weights,
                     m.route);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  e = bf16 ? launch_product_type<true>(false, gate_up_gpc, a, m, stream)
           : launch_product_type<false>(false, gate_up_gpc, a, m, stream);
  if (e != hipSuccess) return e;
  return bf16 ? launch_product_type<true>(true, down_gpc, a, m, stream)
              : launch_product_type<false>(true, down_gpc, a, m, stream);
}

}  // namespace wq
