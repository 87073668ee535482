// A whole mixture-of-experts layer of a few tokens (wq_moe_layer): routing, the chosen
// experts' gate/up projections with SwiGLU, their down projections and the weighted sum.
//
// The layer reads every chosen expert's weights once and does 2 * (rows per expert) products
// per weight, so a large one is bound by the weight stream and a small one by its launches,
// each of which needs the whole result of the one before it.  Nothing is done on the host:
//  1. router_kernel: the logits x router^T.
//  2. route_kernel, one work-group: the tokens' top-k, and for each expert that any token
//     chose (a "slot") its rows.  (Taken in every work-group of the next kernel instead, the
//     routing cost 4 to 30 us more than this launch.)  It forms one token's logits of a
//     small router too.
//  3. product_kernel on the gate/up bank: a work-group per slot and pair of 16-column blocks,
//     a gate and an up block, ends in the activation silu(g) * u.  The grid has room for the
//     most slots there can be; work-groups past the last one end at once.
//  4. product_kernel on the down bank: the same over two neighbouring blocks, ends in fp32
//     rows, one for each (token, choice).
//  5. combine_kernel: each token's rows times their routing weights, in the order of choice
//     (no atomics), and the residual.
// Where there are few weights down_all_kernel does 4 and 5 in one launch.
// Products are 16x16x32 MFMAs on codes dequantized in registers (wq_device.h); each scale
// unit's partial is scaled in fp32.  The activation goes from one product to the next as two
// bf16 values, high + low, for either element type: fp32's range, and 16 bits of it, so that
// y's rounding is the only one that shows (rounded to the element type instead, y was off by 1.4
// times as much, and an fp16 activation past 65504 was infinite).  Codes and E4M3 values are
// exact in bf16.
//
// Measured as a graph, 128-row groups, K x N of an expert 4096 x 2 * 14336 and 14336 x 4096: one
// token of two experts, fp16, 44 us, 4.1 TB/s (products 24.1 us at 5.0 TB/s and 13.5 at 4.5 in a
// kernel trace, routing 5.2, combine 3.8), with E4M3 weights 68 us, 5.3 TB/s (38.5 at 6.2, 21.0 at
// 5.7); four tokens of five to six experts, bf16 with zero points, 99 us, 5.2 TB/s (57.5 us at 6.0,
// 36.8 at 4.7).  16 tokens over 56 of 64 experts of 2048 x 2 * 1024, 64-row groups, 50 us, 3.8 TB/s
// (24.4 us at 5.2, 15.9 at 3.9).
#include <type_traits>

#include "wq_decode.h"
#include "wq_device.h"

namespace wq {
namespace {

constexpr int kMaxT = WQ_MOE_MAX_TOKENS;
constexpr int kMaxE = WQ_MOE_MAX_EXPERTS;

// The routing of a call, in the workspace.  A slot's row is a (token, choice) pair: its number
// token * top_k + choice in the low half, the token in the high half.
struct RouteSlot {
  int32_t expert, rows;  // ascending experts; no rows: past the last chosen expert
  uint32_t pair[kMaxT];
  // by token, for down_all_kernel: its pair here (-1: it has none) and that pair's weight
  int32_t token_pair[kMaxT];
  float token_w[kMaxT];
};
struct Route {
  int32_t used, pad[3];  // slots with rows
  RouteSlot slot[kMaxE];
  float w[kMaxT * WQ_MOE_MAX_TOPK];  // routing weight of each pair
};

struct Bank {
  const u32x4* b;
  const uint16_t* s;
  const uint32_t* z;
  long b_stride, s_stride, z_stride;  // in elements of the above
};

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// ---- routing ---------------------------------------------------------------------------

constexpr int kRouterThreads = 256;

// Products of one expert's router row with T = 1 or 4 tokens (past the last: the last one), over
// k0, k0 + step, ... of the hidden size, 8 elements each; lanes 64 / T * j, ... of the wave return
// token t0 + j's sum over the wave.  Sums and logits are fp64 up to the choice: the order of nearly
// equal logits decides which experts run.  Products are exact, of fp16 values in fp32 (one
// conversion less), of bf16 ones in fp64, whose range they need.
template <bool BF16, int T, int UNROLL>
__device__ __forceinline__ double wave_logits(const uint16_t* x, int ldx, const uint16_t* rp,
                                              int tokens, int t0, int k0, int step, int end,
                                              int lane) {
  using A = Act<BF16>;
  const auto value = [](u32x4 w, int i) {
    return A::value((uint16_t)(w[i / 2] >> (16 * (i % 2))));
  };
  constexpr int N = 4 / T;  // sums of a token, so that four are on their way
  double sums[T][N] = {};
#pragma unroll UNROLL
  for (int k = k0; k < end; k += step) {
    const u32x4 r = *reinterpret_cast<const u32x4*>(rp + k);
    u32x4 xv[T];
#pragma unroll
    for (int j = 0; j < T; ++j)
      xv[j] = *reinterpret_cast<const u32x4*>(x + (long)min(t0 + j, tokens - 1) * ldx + k);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < T; ++j)
        sums[j][i % N] = BF16 ? __builtin_fma((double)value(r, i), (double)value(xv[j], i),
                                              sums[j][i % N])
                              : sums[j][i % N] + (double)(value(r, i) * value(xv[j], i));
  }
  double acc[T];
#pragma unroll
  for (int j = 0; j < T; ++j) {
    acc[j] = sums[j][0];
#pragma unroll
    for (int i = 1; i < N; ++i) acc[j] += sums[j][i];
  }
  double v = acc[0];
  if constexpr (T == 4) {
    // Each exchange halves the tokens a lane carries: token 2 * up + odd is left.
    const bool up = lane & 32, odd = lane & 16;
    const double a0 = (up ? acc[2] : acc[0]) + __shfl_xor(up ? acc[0] : acc[2], 32);
    const double a1 = (up ? acc[3] : acc[1]) + __shfl_xor(up ? acc[1] : acc[3], 32);
    v = (odd ? a1 : a0) + __shfl_xor(odd ? a0 : a1, 16);
  }
#pragma unroll
  for (int d = 32 / T; d >= 1; d /= 2) v += __shfl_xor(v, d);
  return v;
}

// Logits of one expert and four tokens per work-group, whose threads share the hidden size: 2.1 to
// 4.8 us, a launch and a trip to memory, where one CU reading a router of 64 KiB takes 2 us longer
// and one of 256 KiB 10 us.
template <bool BF16>
__global__ __launch_bounds__(kRouterThreads) void router_kernel(
    const uint16_t* __restrict__ x, int ldx, const uint16_t* __restrict__ router, int tokens,
    int n_expert, int hidden, double* __restrict__ logits) {
  __shared__ double red[kRouterThreads / 64][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.x;
  const int t0 = blockIdx.y * 4;
  const double v = wave_logits<BF16, 4, 2>(x, ldx, router + (long)e * hidden, tokens, t0, tid * 8,
                                        kRouterThreads * 8, hidden, lane);
  if ((lane & 15) == 0) red[wave][lane >> 4] = v;
  __syncthreads();
  if (tid < 4 && t0 + tid < tokens) {
    double sum = red[0][tid];
#pragma unroll
    for (int w = 1; w < kRouterThreads / 64; ++w) sum += red[w][tid];
    logits[(t0 + tid) * n_expert + e] = sum;
  }
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  const uint32_t other = __builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xf, 0xf, false);
  return other > x ? other : x;
}

// Maximum over the wave, as a scalar.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = dpp_max<0x111>(x);  // row_shr 1, 2, 4, 8: lane 15 of each row of 16 has its maximum
  x = dpp_max<0x112>(x);
  x = dpp_max<0x114>(x);
  x = dpp_max<0x118>(x);
  x = dpp_max<0x142>(x);  // row_bcast 15 and 31: lane 63 has the wave's
  x = dpp_max<0x143>(x);
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

__device__ __forceinline__ uint64_t read_lane(uint64_t x, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
}

// One token's top-k by its wave: lane j ends with the j-th best expert and its weight.  Equal
// logits go to the lower expert, NaN below everything; PER experts a lane.
template <int PER>
__device__ __forceinline__ void token_top_k(const double* logits, int n_expert, int top_k,
                                            bool renormalize, float routed_scale, int lane,
                                            int& my_id, float& my_w) {
  double l[PER];
  uint64_t key[PER];  // ordered as the logits are; 0 is below every expert's
  bool bad = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < n_expert ? logits[e] : -INFINITY;
    bad |= l[i] != l[i] || l[i] == INFINITY;
    const uint64_t bits = __builtin_bit_cast(uint64_t, l[i] + 0.);  // -0 and 0 are equal
    key[i] = (bits >> 63) ? ~bits : bits | 1ull << 63;
    if (l[i] != l[i]) key[i] = 1;
    if (e >= n_expert) key[i] = 0;
  }
  const bool nan_row = __ballot(bad) != 0;
  // The upper halves of the keys decide, unless two are equal.
  const auto upper = [&](int i) { return (uint32_t)(key[i] >> 32); };
  uint64_t my_key = 0;
  bool done = false;
  if (PER == 1 && n_expert < 4 * top_k) {
    // An expert's place is the number of experts before it: larger keys, and equal ones of
    // lower number.  No round waits for the one before, but there are as many steps as experts,
    // where the rounds below are as many as choices (16 tokens, us for a layer, counted and in
    // rounds: 8 of 8 experts 13.4, 14.5; 4 of 16 14.2, 14.2; 8 of 64 19.0, 18.2; 1 of 64 15.6,
    // 13.4).
    int place = 0;
    const uint64_t full = (uint64_t)upper(0) << 32 | (uint32_t)(63 - lane);
    for (int e0 = 0; e0 < n_expert; e0 += 8) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int e = e0 + k;  // past n_expert the keys are 0
        const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)upper(0), e);
        place += ((uint64_t)other << 32 | (uint32_t)(63 - e)) > full;
      }
    }
    // lane j fetches the key and number of the expert in place j (lanes past the last expert
    // have the places past its, in their order)
    const uint32_t high = __builtin_amdgcn_ds_permute(4 * place, (int)upper(0));
    const uint32_t low = __builtin_amdgcn_ds_permute(4 * place, (int)key[0]);
    my_id = __builtin_amdgcn_ds_permute(4 * place, lane);
    my_key = (uint64_t)high << 32 | low;
    const uint32_t before = __shfl_up(high, 1);
    done = __ballot(lane > 0 && lane <= top_k && high == before) == 0;
  }
  if (!done) {
    for (int j = 0; j < top_k; ++j) {
      uint32_t best = upper(0);
#pragma unroll
      for (int i = 1; i < PER; ++i) best = max(best, upper(i));
      best = wave_max(best);
      unsigned long long has[PER];
      int equal = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        has[i] = __ballot(upper(i) == best);
        equal += __popcll(has[i]);
      }
      if (equal > 1) {
        uint32_t low = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) low = max(low, upper(i) == best ? (uint32_t)key[i] : 0u);
        low = wave_max(low);
#pragma unroll
        for (int i = 0; i < PER; ++i)
          has[i] = __ballot(upper(i) == best && (uint32_t)key[i] == low);
      }
      int id = 0;  // lowest expert with this key
#pragma unroll
      for (int i = PER - 1; i >= 0; --i)
        if (has[i]) id = 64 * i + __builtin_ctzll(has[i]);
      uint64_t chosen = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (id / 64 == i) chosen = read_lane(key[i], id % 64);
      if (lane == j) {
        my_key = chosen;
        my_id = id;
      }
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (id == lane + 64 * i) key[i] = 0;
    }
  }
  const auto value = [](uint64_t k) {
    return __builtin_bit_cast(double, (k >> 63) ? k & ~(1ull << 63) : ~k);
  };
  // (differences are taken in fp64, so that large logits keep small ones)
  const double top = value(read_lane(my_key, 0));
  const float mine = lane < top_k ? expf((float)(value(my_key) - top)) : 0.f;
  float sum = mine;
  if (!renormalize) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += expf((float)(l[i] - top));
  }
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) sum += __shfl_xor(sum, d);
  // no softmax of a row with NaN, or without a logit above -inf
  my_w = nan_row || !(sum > 0.f) ? __builtin_nanf("") : mine / sum * routed_scale;
}

struct RouteArgs {
  const double* logits;
  Route* route;
  int32_t* ids;
  float* weights;
  int tokens, n_expert, top_k, renormalize, slots;  // slots: of the next kernels' grids
  float routed_scale;
  int by_token;  // the slots' token_pair and token_w are needed
  // with the logits formed here:
  const uint16_t *x, *router;
  int ldx, hidden;
};

// One work-group, a wave per token; 5.2 us for one token of 8 experts with the logits of 4096
// elements, 4.6 for 16 of 64 without: a chain of trips to memory and LDS.  PER: 64 experts for each
// lane of a wave, 1 or 4.  ROUTER: 16 waves form one token's logits here too, first (1: fp16, 2:
// bf16): an expert for each, or with fewer of these a part of the hidden size.
template <int PER, int ROUTER>
__global__ __launch_bounds__(kMaxT * 64) void route_kernel(RouteArgs p) {
  __shared__ uint32_t mask_lds[kMaxE];
  __shared__ uint8_t slot_of[kMaxE];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int i = tid; i < kMaxE; i += blockDim.x) mask_lds[i] = 0;
  const double* logits = p.logits;
  if constexpr (ROUTER != 0) {
    __shared__ double part_lds[kMaxT], logit_lds[kMaxT];
    const int segs = kMaxT / p.n_expert;
    if (wave < p.n_expert * segs) {
      const int e = wave / segs, k0 = (wave - e * segs) * 512 + lane * 8;
      const double v = wave_logits<ROUTER == 2, 1, 4>(p.x, p.ldx, p.router + (long)e * p.hidden, 1,
                                                      0, k0, segs * 512, p.hidden, lane);
      if (lane == 0) part_lds[wave] = v;
    }
    __syncthreads();
    if (tid < p.n_expert) {
      double sum = 0.;
      for (int k = 0; k < segs; ++k) sum += part_lds[tid * segs + k];
      logit_lds[tid] = sum;
    }
    logits = logit_lds;
  }
  __syncthreads();
  int id = 0;  // lane j of wave t: token t's j-th choice
  float w = 0.f;
  const bool mine = wave < p.tokens && lane < p.top_k;
  const int pair = wave * p.top_k + lane;
  if (wave < p.tokens) {
    token_top_k<PER>(logits + wave * p.n_expert, p.n_expert, p.top_k, p.renormalize,
                     p.routed_scale, lane, id, w);
    if (mine) {
      atomicOr(&mask_lds[id], 1u << wave);
      p.route->w[pair] = w;
      if (p.ids != nullptr) p.ids[pair] = id;
      if (p.weights != nullptr) p.weights[pair] = w;
    }
  }
  __syncthreads();
  if (wave == 0) {
    int slots = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t m = mask_lds[64 * i + lane];
      const unsigned long long act = __ballot(m != 0);
      const int slot = slots + __popcll(act & ((1ull << lane) - 1));
      slots += __popcll(act);
      if (m != 0) {
        slot_of[64 * i + lane] = (uint8_t)slot;
        p.route->slot[slot].expert = 64 * i + lane;
        p.route->slot[slot].rows = __popc(m);
      }
    }
    for (int i = slots + lane; i < p.slots; i += 64) p.route->slot[i].rows = 0;
    if (lane == 0) p.route->used = slots;
  }
  if (p.by_token) {  // no pairs first (p.slots are at least as many as the slots with rows)
    for (int i = tid; i < p.slots * kMaxT; i += blockDim.x)
      p.route->slot[i / kMaxT].token_pair[i % kMaxT] = -1;
  }
  __syncthreads();
  if (mine) {  // the expert's rows lie in token order
    RouteSlot& slot = p.route->slot[slot_of[id]];
    slot.pair[__popc(mask_lds[id] & ((1u << wave) - 1))] = (uint32_t)pair | (uint32_t)wave << 16;
    if (p.by_token) {
      slot.token_pair[wave] = pair;
      slot.token_w[wave] = w;
    }
  }
}

// Orders a wave's own LDS accesses (they execute in order; this keeps the compiler to it).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ---- the quantized products ------------------------------------------------------------

// bf16 has no packed subtract, so its codes enter the products as 128 + q (one mask-and-or a
// pair) and (128 + z) times the rows' sums is taken off each unit's partial; the sums are a
// product with ones, on a matrix unit that has the time.  fp16 codes are made exact.
template <bool BF16, bool W8>
constexpr bool kBiased = BF16 && !W8;

// 16 rows of a 128-row chunk as the A operands of its four 32-row steps, in PARTS parts that are
// added: one, or the activation's two.
template <int PARTS>
struct Rows {
  f16x8 v[PARTS][4];
};

// The sums of a 128-row chunk of activations over each scale unit, as the products lay them.
template <bool BF16, bool W8, int GPC>
struct RowSums {
  f32x4 v[kBiased<BF16, W8> ? GPC : 1];

  template <int PARTS>
  __device__ __forceinline__ void form(const Rows<PARTS>& a, int lane) {
    if constexpr (kBiased<BF16, W8>) {
      using A = Act<true>;
      const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
      const u32x4 one_bits = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
      const bf16x8 ones = __builtin_bit_cast(bf16x8, one_bits), none{};
      if constexpr (GPC <= 4) {
#pragma unroll
        for (int u = 0; u < GPC; ++u) {
          v[u] = zero;
#pragma unroll
          for (int j = 4 / GPC * u; j < 4 / GPC * (u + 1); ++j)
#pragma unroll
            for (int i = 0; i < PARTS; ++i) v[u] = A::mfma16(a.v[i][j], ones, v[u]);
        }
      } else {
        const bool second = lane >= 32;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = v[2 * j + 1] = zero;
#pragma unroll
          for (int i = 0; i < PARTS; ++i) {
            v[2 * j] = A::mfma16(a.v[i][j], second ? none : ones, v[2 * j]);
            v[2 * j + 1] = A::mfma16(a.v[i][j], second ? ones : none, v[2 * j + 1]);
          }
        }
      }
    }
  }
};

// One 128-row chunk of a 16-column block as its wave holds it: codes, scales, zero points.
// BF16: of the scales; OPS: of the products' operands.
template <bool BF16, bool OPS, bool W8, bool ZP, int GPC>
struct Chunk {
  using A = Act<OPS>;
  using Sums = RowSums<OPS, W8, GPC>;
  u32x4 w[W8 ? 2 : 1];
  uint16_t s[GPC];
  uint32_t z[ZP ? GPC : 1];  // the lane's half of the unit's codes

  // at: chunk index of the expert's layout (block * groups + group)
  __device__ __forceinline__ void load(const u32x4* b, const uint16_t* sp, const uint32_t* zp,
                                       long at, int lane) {
#pragma unroll
    for (int v = 0; v < (W8 ? 2 : 1); ++v)
      w[v] = __builtin_nontemporal_load(b + (at * (W8 ? 2 : 1) + v) * 64 + lane);
#pragma unroll
    for (int u = 0; u < GPC; ++u) s[u] = sp[(at * GPC + u) * 16 + (lane & 15)];
    if constexpr (ZP) {
#pragma unroll
      for (int u = 0; u < GPC; ++u) z[u] = zp[(at * GPC + u) * 2 + ((lane >> 3) & 1)];
    }
  }

  // acc += a x chunk
  template <int PARTS>
  __device__ __forceinline__ void multiply(const Rows<PARTS>& a, const Sums& sums, int lane,
                                           f32x4& acc) const {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const auto step = [&](int j, typename A::W8 w, f32x4 part) {
#pragma unroll
      for (int i = 0; i < PARTS; ++i) part = A::mfma16(a.v[i][j], w, part);
      return part;
    };
    const auto code = [&](int u) {
      return ZP ? (int)((z[ZP ? u : 0] >> (4 * (lane & 7))) & 0xFu) : 8;
    };
    const auto add = [&](int u, f32x4 part) {
      const float f = Act<BF16>::value(s[u]);
      if constexpr (kBiased<OPS, W8>) {
        const float excess = (float)(128 + code(u));
#pragma unroll
        for (int e = 0; e < 4; ++e) part[e] = __builtin_fmaf(-excess, sums.v[u][e], part[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(f, part[e], acc[e]);
    };
    if constexpr (W8) {
      f32x4 p = zero;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        p = step(j, A::fp8(w[j / 2][2 * (j % 2)], w[j / 2][2 * (j % 2) + 1]), p);
      add(0, p);
    } else {
      // the weights of step j, as unit u's zero point makes them
      const auto weights = [&](int j, int u) -> typename A::W8 {
        if constexpr (OPS)
          return dequant8_bf_biased(w[0][j], magic_reg_bf128());
        else
          return A::dequant(w[0][j], A::zero(code(u)), A::magic());
      };
      if constexpr (GPC <= 4) {
#pragma unroll
        for (int u = 0; u < GPC; ++u) {
          f32x4 p = zero;
#pragma unroll
          for (int j = 4 / GPC * u; j < 4 / GPC * (u + 1); ++j) p = step(j, weights(j, u), p);
          add(u, p);
        }
      } else {
        // 16-row units: lanes 0-31 hold a step's first unit, lanes 32-63 its second; each
        // unit has its product, the other half's weights set to zero
        const bool second = lane >= 32;
        const typename A::W8 none{};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const typename A::W8 q0 = weights(j, 2 * j), q1 = weights(j, 2 * j + 1);
          add(2 * j, step(j, second ? none : q0, zero));
          add(2 * j + 1, step(j, second ? q1 : none, zero));
        }
      }
    }
  }
};

struct ProductArgs {
  const uint16_t* a;  // x, rows by token; or the activation, rows by pair
  Bank bank;
  const Route* route;
  uint16_t* h;   // GATE_UP: the activation [pair][high, low][inter]
  float* part;   // else: fp32 rows [pair][hidden]
  long lda;
  int groups, n;  // n: columns of a row of the output
};

// Two neighbouring 16-column blocks of a slot's expert.  Each wave takes a run of 128-row
// groups, GW at a time, with all of their weights requested at once.  A lane's activations
// serve both blocks; up to kStagedLines lines (a load a lane for each group in flight) the wave
// first brings into LDS, in whole lines: 16 rows read as MFMA operands are as many loads
// as the weights of both blocks, and operands held in registers leave none for weights in flight
// (the three layers above without staging 46.0, 117 and 57.8 us, with it 44.1, 103 and 51.1;
// twice the lines of the activation staged: 43.1, 101 and 49.7 us against 42.7, 98.0 and 49.6).
constexpr int kStagedLines = 4;

// Groups in flight, by the registers of a chunk: codes, scales, zero points.  (Layers of 1 token,
// two and four groups, us: 5 registers 44.9 and 43.3, 8 48.5 and 47.8, 12 with zero points 55.1 and
// 57.9, 12 without 74.2 and 76.9, 20 98.2 and 107.4; E4M3, 9: 66.8 and 65.9.)
template <bool W8, bool ZP, int GPC>
constexpr int kInFlight = (W8 ? 8 : 4) + GPC * (ZP ? 2 : 1) <= 9 ? 4 : 2;

template <bool GATE_UP, bool BF16, bool W8, bool ZP, int GPC, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void product_kernel(ProductArgs p) {
  constexpr int PARTS = GATE_UP ? 1 : 2;  // lines of a row: the activation has two
  using C = Chunk<BF16, BF16 || !GATE_UP, W8, ZP, GPC>;
  constexpr int GW = kInFlight<W8, ZP, GPC>;
  constexpr int LR = GW * 16 + 1;  // granules of a staged line, one of padding
  constexpr int kStage = WAVES * kStagedLines * LR * 16, kRed = 2 * WAVES * 64 * 16;
  __shared__ __align__(16) uint8_t lds[kStage > kRed ? kStage : kRed];
  const RouteSlot& slot = p.route->slot[blockIdx.y];
  const int expert = slot.expert, rows = slot.rows;
  if (rows == 0) return;  // past the last chosen expert
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, qd = lane >> 4;
  const uint32_t row_pair = slot.pair[row];  // (not written past the slot's rows)
  // rows past the last repeat the first (and are not stored)
  // (read from the first lane by the whole wave, not inside the choice between the two)
  const uint32_t first_pair = (uint32_t)__builtin_amdgcn_readfirstlane((int)row_pair);
  const uint32_t pair = row < rows ? row_pair : first_pair;
  const auto row_at = [&](uint32_t pr) {
    return p.a + (long)(GATE_UP ? pr >> 16 : pr & 0xffffu) * PARTS * p.lda;
  };
  const u32x4* b = p.bank.b + expert * p.bank.b_stride;
  const uint16_t* s = p.bank.s + expert * p.bank.s_stride;
  const uint32_t* z = ZP ? p.bank.z + expert * p.bank.z_stride : nullptr;

  // Up to eight rows of two lines are the 16 rows of one product, which are added in pairs at the
  // end; more rows take a product for each line (rows of two products 45.0, 107 and 51.1 us for
  // the three layers above).
  const bool paired = PARTS == 2 && rows <= 8;
  const long block0 = 2L * blockIdx.x * p.groups, block1 = block0 + p.groups;
  f32x4 acc0 = {0.f, 0.f, 0.f, 0.f}, acc1 = acc0;
  const int last = p.groups * (wave + 1) / WAVES;
  int g0 = p.groups * wave / WAVES;
  const int lines = rows * PARTS;
  if (lines <= kStagedLines) {
    u32x4* const own = reinterpret_cast<u32x4*>(lds) + wave * kStagedLines * LR;
    const u32x4* ap = own + (row < lines ? row : 0) * LR + qd;
    for (; g0 < last; g0 += GW) {
      const int n = min(GW, last - g0);
      u32x4 stage[GW];
#pragma unroll
      for (int u = 0; u < GW; ++u) {  // 64 granules of the lines' GW * 16 each
        if (u * 64 < lines * GW * 16) {
          const int i = u * 64 + lane, c = i % (GW * 16);
          const int line = min(i / (GW * 16), lines - 1);
          const uint32_t pr = __shfl(pair, line / PARTS);
          stage[u] = reinterpret_cast<const u32x4*>(row_at(pr) + line % PARTS * p.lda +
                                                    (long)g0 * kGroup)[min(c, n * 16 - 1)];
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // the rows are requested before any weight
      C c0[GW], c1[GW];
#pragma unroll
      for (int i = 0; i < GW; ++i) {
        const int g = g0 + min(i, n - 1);
        c0[i].load(b, s, z, block0 + g, lane);
        c1[i].load(b, s, z, block1 + g, lane);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < GW; ++u) {
        if (u * 64 < lines * GW * 16) {
          const int i = u * 64 + lane;
          own[i / (GW * 16) * LR + i % (GW * 16)] = stage[u];
        }
      }
      wave_lds_fence();
#pragma unroll
      for (int i = 0; i < GW; ++i) {
        if (i >= n) continue;
        Rows<1> a;
#pragma unroll
        for (int j = 0; j < 4; ++j) a.v[0][j] = __builtin_bit_cast(f16x8, ap[16 * i + 4 * j]);
        typename C::Sums sums;
        sums.form(a, lane);
        c0[i].multiply(a, sums, lane, acc0);
        c1[i].multiply(a, sums, lane, acc1);
      }
      wave_lds_fence();
    }
  } else {
    constexpr int U = GW >= 2 ? 2 : 1;
    const auto direct = [&](auto parts, const uint16_t* ap) {
      constexpr int P = decltype(parts)::value;
      for (; g0 < last; g0 += U) {
        C c0[U], c1[U];
        Rows<P> a[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int g = min(g0 + i, last - 1);
          c0[i].load(b, s, z, block0 + g, lane);
          c1[i].load(b, s, z, block1 + g, lane);
#pragma unroll
          for (int k = 0; k < P; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              a[i].v[k][j] =
                  *reinterpret_cast<const f16x8*>(ap + k * p.lda + (long)g * kGroup + 32 * j);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (g0 + i >= last) continue;
          typename C::Sums sums;
          sums.form(a[i], lane);
          c0[i].multiply(a[i], sums, lane, acc0);
          c1[i].multiply(a[i], sums, lane, acc1);
        }
      }
    };
    if (paired)
      direct(std::integral_constant<int, 1>(),
             row_at(__shfl(pair, row / 2)) + row % 2 * p.lda + 8 * qd);
    else
      direct(std::integral_constant<int, PARTS>(), row_at(pair) + 8 * qd);
  }
  __syncthreads();  // the staged rows are no longer read
  f32x4(*const red)[WAVES][64] = reinterpret_cast<f32x4(*)[WAVES][64]>(lds);
  if (paired) {  // lines 2 r and 2 r + 1 lie in neighbouring elements of a lane
    const int at = qd / 2 * 16 + row, e = 2 * (qd % 2);
    float* const r0 = reinterpret_cast<float*>(&red[0][wave][at]) + e;
    float* const r1 = reinterpret_cast<float*>(&red[1][wave][at]) + e;
    r0[0] = acc0[0] + acc0[1];
    r0[1] = acc0[2] + acc0[3];
    r1[0] = acc1[0] + acc1[1];
    r1[1] = acc1[2] + acc1[3];
  } else {
    red[0][wave][lane] = acc0;
    red[1][wave][lane] = acc1;
  }
  __syncthreads();
  // the lane's four elements of the two blocks are summed by different waves, in wave order
#pragma unroll
  for (int e = wave; e < 4; e += WAVES) {
    const int r = 4 * qd + e;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      s0 += reinterpret_cast<const float*>(&red[0][w][lane])[e];
      s1 += reinterpret_cast<const float*>(&red[1][w][lane])[e];
    }
    const long out = (long)(__shfl(pair, r) & 0xffffu) * p.n;
    if (r < rows) {
      if constexpr (GATE_UP) {
        const float v = silu_times(s0, s1);
        const uint16_t high = Act<true>::round(v);
        const float left = v - Act<true>::value(high);  // exact
        uint16_t* const h = p.h + 2 * out + 16 * blockIdx.x + row;
        h[0] = high;
        h[p.n] = left - left == 0.f ? Act<true>::round(left) : 0;  // none beside inf or NaN
      } else {
        p.part[out + 32 * blockIdx.x + row] = s0;
        p.part[out + 32 * blockIdx.x + 16 + row] = s1;
      }
    }
  }
}

struct DownArgs {
  const uint16_t* h;  // the activation [pair][high, low][inter]
  Bank bank;
  const Route* route;
  const uint16_t* residual;
  uint16_t* y;
  int inter, groups, tokens, ldr, ldy;
};

// The down projections of a small layer with the weighted sum: a work-group per 16-column block
// of the output, whose waves share all slots' 128-row groups.  The rows are the tokens; one that
// did not choose a slot's expert has zeros there, and its products (of a zero, and of whatever
// that expert's weights are) are left out.  Bound by three trips to memory one after the other:
// the slot, its rows and weights, the store.  Two groups in flight, fewer waves, or the slots'
// rows brought to LDS first were no faster.
constexpr int kDownWaves = 16;

template <bool BF16, bool W8, bool ZP, int GPC>
__global__ __launch_bounds__(kDownWaves * 64) void down_all_kernel(DownArgs p) {
  using A = Act<BF16>;
  using C = Chunk<BF16, true, W8, ZP, GPC>;
  __shared__ f32x4 red[kDownWaves][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = lane & 15, qd = lane >> 4;
  const int items = p.route->used * p.groups;
  const int last = items * (wave + 1) / kDownWaves;
  const long block = (long)blockIdx.x * p.groups;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int i = items * wave / kDownWaves; i < last; ++i) {
    const int s = i / p.groups, g = i - s * p.groups;
    const RouteSlot& slot = p.route->slot[s];
    const long e = slot.expert;
    C c;
    c.load(p.bank.b + e * p.bank.b_stride, p.bank.s + e * p.bank.s_stride,
           ZP ? p.bank.z + e * p.bank.z_stride : nullptr, block + g, lane);
    const int pair = slot.token_pair[row];
    const uint16_t* ap = p.h + 2L * max(pair, 0) * p.inter + (long)g * kGroup + 8 * qd;
    Rows<2> a;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a.v[k][j] = *reinterpret_cast<const f16x8*>(ap + k * p.inter + 32 * j);
        if (pair < 0) a.v[k][j] = f16x8{};
      }
    int member[4];
    float w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      member[k] = slot.token_pair[4 * qd + k];
      w[k] = slot.token_w[4 * qd + k];  // (not written where it has no pair)
    }
    typename C::Sums sums;
    sums.form(a, lane);
    f32x4 part = {0.f, 0.f, 0.f, 0.f};
    c.multiply(a, sums, lane, part);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      acc[k] = member[k] >= 0 ? __builtin_fmaf(w[k], part[k], acc[k]) : acc[k];
  }
  red[wave][lane] = acc;
  __syncthreads();
  // the block's 16 rows of 16 columns, in wave order
  const int t = tid >> 4, col = tid & 15;
  if (t >= p.tokens) return;
  const long at = 16 * blockIdx.x + col;
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < kDownWaves; ++k)
    sum += reinterpret_cast<const float*>(&red[k][16 * (t >> 2) + col])[t & 3];
  if (p.residual != nullptr) sum += A::value(p.residual[(long)t * p.ldr + at]);
  p.y[(long)t * p.ldy + at] = A::round(sum);
}

// y[t] = residual[t] + sum over the token's choices j of w_j part[t][j], 4 columns a thread.
// Bound by its launch and a trip to memory: 3.8 us for one token of 4096, 4.3 for 16 of 2048.
template <bool BF16>
__global__ __launch_bounds__(256) void combine_kernel(const float* __restrict__ part,
                                                      const Route* __restrict__ route, int top_k,
                                                      int hidden, const uint16_t* residual,
                                                      int ldr, uint16_t* y, int ldy) {
  using A = Act<BF16>;
  const int col = 4 * (blockIdx.x * 256 + threadIdx.x);
  const int t = blockIdx.y;
  if (col >= hidden) return;
  u32x2 res = {0u, 0u};
  if (residual != nullptr) res = *reinterpret_cast<const u32x2*>(residual + (long)t * ldr + col);
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < top_k; j0 += 4) {  // four rows requested together
    float w[4];
    f32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = t * top_k + min(j0 + i, top_k - 1);
      w[i] = route->w[pair];
      v[i] = *reinterpret_cast<const f32x4*>(part + (long)pair * hidden + col);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (j0 + i >= top_k) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(w[i], v[i][e], sum[e]);
    }
  }
  uint32_t out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    out[e] = A::round(sum[e] + A::value((uint16_t)(res[e / 2] >> (16 * (e % 2)))));
  *reinterpret_cast<u32x2*>(y + (long)t * ldy + col) =
      u32x2{out[0] | out[1] << 16, out[2] | out[3] << 16};
}

int max_slots(int tokens, int n_expert, int top_k) {
  return tokens * top_k < n_expert ? tokens * top_k : n_expert;
}

Bank bank_of(const wq_expert_bank& b) {
  return Bank{static_cast<const u32x4*>(b.b), static_cast<const uint16_t*>(b.s),
              static_cast<const uint32_t*>(b.zp), (long)(b.b_stride_bytes / 16),
              (long)(b.s_stride_bytes / 2), (long)(b.zp_stride_bytes / 4)};
}

struct MoeScratch {
  double* logits;
  Route* route;
  uint16_t* h;
  float* part;
  size_t bytes;
};

MoeScratch scratch_of(void* base, int tokens, int n_expert, int top_k, int hidden, int inter) {
  const size_t logits = round256((size_t)tokens * n_expert * sizeof(double));
  const size_t route = round256(sizeof(Route));
  const size_t h = round256((size_t)tokens * top_k * inter * 4);
  char* p = static_cast<char*>(base);
  return MoeScratch{reinterpret_cast<double*>(p), reinterpret_cast<Route*>(p + logits),
                    reinterpret_cast<uint16_t*>(p + logits + route),
                    reinterpret_cast<float*>(p + logits + route + h),
                    logits + route + h + (size_t)tokens * top_k * hidden * sizeof(float)};
}

template <bool GATE_UP, bool BF16, bool W8, bool ZP, int GPC>
hipError_t launch_product(const wq_moe_args& a, const MoeScratch& m, hipStream_t stream) {
  ProductArgs p{};
  p.a = GATE_UP ? static_cast<const uint16_t*>(a.x) : m.h;
  p.bank = bank_of(GATE_UP ? a.gate_up : a.down);
  p.route = m.route;
  p.h = m.h;
  p.part = m.part;
  p.lda = GATE_UP ? a.ldx : a.inter;
  p.groups = (GATE_UP ? a.hidden : a.inter) / kGroup;
  p.n = GATE_UP ? a.inter : a.hidden;
  const dim3 grid(GATE_UP ? a.inter / 16 : a.hidden / 32,
                  max_slots(a.tokens, a.n_expert, a.top_k));
#define WQ_MOE_PRODUCT(W)                                                                      \
  hipLaunchKernelGGL((product_kernel<GATE_UP, BF16, W8, ZP, GPC, W>), grid, dim3(W * 64), 0,   \
                     stream, p)
  // Four waves; eight where each would have a long run and there are few work-groups (down
  // projection of 112 groups, 1 token: 45.9 -> 42.8 us for the layer; 64 groups and fewer are
  // slower with eight: 16 tokens of 64 experts, 50.4 -> 61.9 us).
  // Two for a short K when there are many work-groups (8 groups, 64 slots: 50.4 -> 48.5 us; 8
  // slots: 18.1 -> 18.8).
  if (p.groups <= 8 && grid.y > 8)
    WQ_MOE_PRODUCT(2);
  else if (p.groups <= 64)
    WQ_MOE_PRODUCT(4);
  else
    WQ_MOE_PRODUCT(8);
#undef WQ_MOE_PRODUCT
  return hipGetLastError();
}

template <bool BF16, bool W8, bool ZP, int GPC>
hipError_t launch_down_all(const wq_moe_args& a, const MoeScratch& m, hipStream_t stream) {
  const DownArgs p{m.h,
                   bank_of(a.down),
                   m.route,
                   static_cast<const uint16_t*>(a.residual),
                   static_cast<uint16_t*>(a.y),
                   a.inter,
                   a.inter / kGroup,
                   a.tokens,
                   a.ldr,
                   a.ldy};
  hipLaunchKernelGGL((down_all_kernel<BF16, W8, ZP, GPC>), dim3(a.hidden / 16),
                     dim3(kDownWaves * 64), 0, stream, p);
  return hipGetLastError();
}

// DOWN_ALL: down_all_kernel, else product_kernel.
template <bool GATE_UP, bool DOWN_ALL, bool BF16, bool W8, bool ZP, int GPC>
hipError_t launch_bank(const wq_moe_args& a, const MoeScratch& m, hipStream_t stream) {
  if constexpr (DOWN_ALL)
    return launch_down_all<BF16, W8, ZP, GPC>(a, m, stream);
  else
    return launch_product<GATE_UP, BF16, W8, ZP, GPC>(a, m, stream);
}

template <bool GATE_UP, bool DOWN_ALL, bool BF16>
hipError_t launch_bank_type(int gpc, const wq_moe_args& a, const MoeScratch& m,
                            hipStream_t stream) {
  if (a.flags & WQ_FLAG_FP8)
    return launch_bank<GATE_UP, DOWN_ALL, BF16, true, false, 1>(a, m, stream);
  const bool zp = (a.flags & WQ_FLAG_HAS_ZP) != 0;
  switch (gpc) {
#define WQ_MOE_GPC(G)                                                                    \
  case G:                                                                                \
    return zp ? launch_bank<GATE_UP, DOWN_ALL, BF16, false, true, G>(a, m, stream)       \
              : launch_bank<GATE_UP, DOWN_ALL, BF16, false, false, G>(a, m, stream)
    WQ_MOE_GPC(1);
    WQ_MOE_GPC(2);
    WQ_MOE_GPC(4);
    WQ_MOE_GPC(8);
#undef WQ_MOE_GPC
    default: return hipErrorInvalidValue;
  }
}

template <bool BF16>
hipError_t launch_route(const wq_moe_args& a, const MoeScratch& m, bool by_token,
                        hipStream_t stream) {
  RouteArgs p{};
  p.logits = m.logits;
  p.route = m.route;
  p.ids = a.ids;
  p.weights = a.weights;
  p.tokens = a.tokens;
  p.n_expert = a.n_expert;
  p.top_k = a.top_k;
  p.renormalize = a.renormalize;
  p.slots = max_slots(a.tokens, a.n_expert, a.top_k);
  p.routed_scale = a.routed_scale;
  p.by_token = by_token;
  p.x = static_cast<const uint16_t*>(a.x);
  p.router = static_cast<const uint16_t*>(a.router);
  p.ldx = a.ldx;
  p.hidden = a.hidden;
  // The routing's one work-group forms one token's logits of a small router as well, a launch less
  // (us for the layer, two launches and one, by the router's elements: 8192 11.55, 10.75; 16384
  // 12.1, 11.5; 32768 14.5, 14.1; more, with sums of eight products in fp32, 65536 14.6, 14.3 or
  // 15.1; 131072 18.3, 19.7).  Of several tokens fp64 sums keep one CU for as long as the launch
  // takes (4096 elements and four tokens 11.8, 12.0; 8192 12.2, 12.2).
  if (a.tokens == 1 && a.n_expert <= kMaxT && a.n_expert * a.hidden <= 32768) {
    hipLaunchKernelGGL((route_kernel<1, BF16 ? 2 : 1>), dim3(1), dim3(kMaxT * 64), 0, stream, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((router_kernel<BF16>), dim3(a.n_expert, (a.tokens + 3) / 4),
                     dim3(kRouterThreads), 0, stream, p.x, a.ldx, p.router, a.tokens, a.n_expert,
                     a.hidden, m.logits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 block(64 * a.tokens);
  if (a.n_expert <= 64)
    hipLaunchKernelGGL((route_kernel<1, 0>), dim3(1), block, 0, stream, p);
  else
    hipLaunchKernelGGL((route_kernel<kMaxE / 64, 0>), dim3(1), block, 0, stream, p);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_moe_type(const wq_moe_args& a, int gate_up_gpc, int down_gpc,
                           hipStream_t stream) {
  const MoeScratch m =
      scratch_of(a.workspace, a.tokens, a.n_expert, a.top_k, a.hidden, a.inter);
  // A work-group takes all slots' groups of a column block while that is one for each wave: two
  // launches become one (us, product and combine / down_all: 8 groups 13.0, 12.0; 16 13.6, 13.1;
  // 24 18.9, 19.7; 32 15.9, 16.9 and 18.3, 20.7; 48 17.2, 20.1).
  const bool down_all = max_slots(a.tokens, a.n_expert, a.top_k) * (a.inter / kGroup) <= 16;
  hipError_t e = launch_route<BF16>(a, m, down_all, stream);
  if (e != hipSuccess) return e;
  e = launch_bank_type<true, false, BF16>(gate_up_gpc, a, m, stream);
  if (e != hipSuccess) return e;
  if (down_all) return launch_bank_type<false, true, BF16>(down_gpc, a, m, stream);
  e = launch_bank_type<false, false, BF16>(down_gpc, a, m, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((combine_kernel<BF16>), dim3((a.hidden + 1023) / 1024, a.tokens), dim3(256),
                     0, stream, m.part, m.route, a.top_k, a.hidden,
                     static_cast<const uint16_t*>(a.residual), a.ldr,
                     static_cast<uint16_t*>(a.y), a.ldy);
  return hipGetLastError();
}

}  // namespace

size_t moe_workspace_bytes(int tokens, int n_expert, int top_k, int hidden, int inter) {
  return scratch_of(nullptr, tokens, n_expert, top_k, hidden, inter).bytes;
}

hipError_t launch_moe_layer(const wq_moe_args& a, int gate_up_gpc, int down_gpc,
                            hipStream_t stream) {
  return (a.flags & WQ_FLAG_BF16) ? launch_moe_type<true>(a, gate_up_gpc, down_gpc, stream)
                                  : launch_moe_type<false>(a, gate_up_gpc, down_gpc, stream);
}

}  // namespace wq
