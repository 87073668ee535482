// Norms of the query and key heads, rotary positions and the paged cache write of new tokens
// (wq_norm_rope_append), and the read of a 4-bit cache's slots (wq_cache4_read).
//
// A head lies in the registers of d / 8 lanes (rounded up to a power of two, so that several heads
// share a wave): its sum of squares is an exchange between these lanes, the rotation is a lane's
// own, because a lane holds both halves of four pairs, and everything between the one read and the
// one write is fp32.  For a 4-bit cache the head then goes through LDS once, so that a lane gets
// eight elements in a row: a dword of codes, whose group's smallest and largest value are again an
// exchange between lanes.
//
// Sines and cosines are formed once per work-group and token, the angle in fp64 (a position of
// 10^6 times an fp32 frequency loses the phase in fp32).
//
// Few tokens are bound by their trips to memory (one, 4-bit: 4.0 us), many 4-bit ones by instructions
// (2048 tokens of 32 + 2 x 8 heads of 128, groups of 32: 16.7 us for 46 MB, of which 10 are the issue of
// vector instructions), others by memory (16-bit 12.9 us, 3.9 TB/s, 8192 tokens 45.1 us, 4.5 TB/s).  The
// read of 2048 4-bit tokens takes 5.1 us.
#include <algorithm>
#include <type_traits>

#include "wq_decode.h"
#include "wq_device.h"

namespace wq {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kMaxPairs = 128;  // head_dim <= 256

enum CacheKind { kCache16, kCacheE4m3, kCache4 };

struct AppendArgs {
  const uint16_t *q, *k, *v, *q_norm, *k_norm;
  uint16_t* q_out;
  void *kc, *vc;
  uint32_t *k_pairs, *v_pairs;
  const float *k_scale, *v_scale;
  const int64_t* slots;
  const int32_t* positions;
  const float* inv_freq;
  int64_t page_stride, slot_stride, head_stride;
  int64_t pair_page, pair_slot, pair_head;
  int64_t total_slots;
  int tokens, q_heads, kv_heads, d, half, page_size, group;
  int ldq, ldk, ldv, ldqo;
  int end[WQ_MAX_ROPE_AXES];  // first pair past each axis
  int axes;
  int lanes_log2;             // lanes of a head
  float eps, inv_d;
};

template <bool BF16>
__device__ __forceinline__ void unpack4(u32x2 w, float* f) {
  using A = Act<BF16>;
  f[0] = A::value((uint16_t)w[0]);
  f[1] = A::value((uint16_t)(w[0] >> 16));
  f[2] = A::value((uint16_t)w[1]);
  f[3] = A::value((uint16_t)(w[1] >> 16));
}

template <bool BF16>
__device__ __forceinline__ u32x2 pack4(const float* f) {
  using A = Act<BF16>;
  return u32x2{(uint32_t)A::round(f[0]) | ((uint32_t)A::round(f[1]) << 16),
               (uint32_t)A::round(f[2]) | ((uint32_t)A::round(f[3]) << 16)};
}

// value / scale as E4M3: clamped to the largest finite value (NaN passes), nearest even.
__device__ __forceinline__ uint32_t pack4_e4m3(const float* f, float scale) {
  float c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v = f[i] / scale;
    c[i] = v != v ? v : fminf(fmaxf(v, -448.f), 448.f);
  }
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
  return (uint32_t)w;
}

// (a 64-bit division costs as much as a head's norm)
__device__ __forceinline__ int64_t page_of(int64_t slot, int page_size, int64_t total) {
  return total <= 0xffffffffll ? (int64_t)((uint32_t)slot / (uint32_t)page_size) : slot / page_size;
}

// f over `width` neighbouring lanes, a power of two up to 32: what a step has made equal in a group
// may come from any lane of the neighbouring group, so mirrors serve where no exchange does.
template <class F>
__device__ __forceinline__ float over_lanes(float x, int width, F f) {
  const auto dpp = [&](auto ctrl) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf,
                                           0xf, false));
  };
  if (width > 1) x = f(x, dpp(std::integral_constant<int, 0xB1>()));   // quad_perm 1 0 3 2
  if (width > 2) x = f(x, dpp(std::integral_constant<int, 0x4E>()));   // quad_perm 2 3 0 1
  if (width > 4) x = f(x, dpp(std::integral_constant<int, 0x141>()));  // row_half_mirror
  if (width > 8) x = f(x, dpp(std::integral_constant<int, 0x140>()));  // row_mirror
  if (width > 16) {
    const auto rows = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x),
                                                       __builtin_bit_cast(uint32_t, x), false, false);
    x = f(__builtin_bit_cast(float, (uint32_t)rows[0]), __builtin_bit_cast(float, (uint32_t)rows[1]));
  }
  return x;
}
__device__ __forceinline__ float lanes_sum(float x, int width) {
  return over_lanes(x, width, [](float a, float b) { return a + b; });
}

// Eight elements of a group whose lanes are `width` wide: their codes, and the group's pair.  A
// lane past the head's end takes part with zeros and `in` false.
//
// A quotient is the product q = t / scale by the reciprocal instruction, two steps off at most, plus
// its remainder times the reciprocal.  The scale has 11 bits or fewer, so the remainder t - q scale is
// exact, the sum is off the quotient by 2^-20 of a step before it is rounded, and a quotient of 24
// bits by 11 is nearer than 2^-12 of a step to no border of rounding: the codes are those of a
// division, ties among them, for a third of its instructions.
template <bool BF16>
__device__ __forceinline__ uint32_t quantize8(const float* x, bool in, int width, uint32_t& pair) {
  using A = Act<BF16>;
  float low = x[0], high = x[0], bad = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    low = fminf(low, x[i]);
    high = fmaxf(high, x[i]);
    bad = __builtin_fmaf(x[i], 0x1p-9f, bad);  // not finite for a NaN or an infinity alone
  }
  low = over_lanes(in ? low : INFINITY, width, [](float a, float b) { return fminf(a, b); });
  high = over_lanes(in ? high : -INFINITY, width, [](float a, float b) { return fmaxf(a, b); });
  bad = lanes_sum(bad * 0.f, width);
  uint32_t sbits = A::round((high - low) / 15.f), obits = A::round(low);
  float scale = A::value((uint16_t)sbits);
  const float offset = A::value((uint16_t)obits);
  if (!((scale - scale) + (offset - offset) + bad == 0.f)) {
    sbits = obits = A::round(__builtin_nanf(""));
    scale = 0.f;
  }
  pair = sbits | obits << 16;
  const float inverse = __builtin_amdgcn_rcpf(scale);
  const bool far = scale < 0x1p-90f || scale > 0x1p120f;  // the remainder or t may leave fp32's range
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = x[i] - offset, q = t * inverse;
    c[i] = __builtin_fmaf(__builtin_fmaf(-q, scale, t), inverse, q);
  }
  if (__ballot(far && scale > 0.f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = far ? (x[i] - offset) / scale : c[i];
  }
  float half[2] = {0.f, 0.f};  // four codes each, as a number
#pragma unroll
  for (int i = 7; i >= 0; --i)
    half[i / 4] = __builtin_fmaf(half[i / 4], 16.f, rintf(__builtin_amdgcn_fmed3f(c[i], 0.f, 15.f)));
  const uint32_t codes = (uint32_t)half[0] | (uint32_t)half[1] << 16;
  return scale > 0.f ? codes : 0u;
}

template <bool BF16, int CACHE, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void norm_rope_append_kernel(AppendArgs p) {
  __shared__ __align__(16) float cs[kMaxPairs], sn[kMaxPairs];
  __shared__ __align__(16) float rows[CACHE == kCache4 ? kWaves : 1][64 * 8];
  const int token = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lanes = 1 << p.lanes_log2, per_wave = 64 >> p.lanes_log2;
  const int e = lane & (lanes - 1);
  const int per_head = p.d / 8, turned = p.half / 4;  // units of eight elements; turned ones
  const int heads = p.q_heads + 2 * p.kv_heads;
  const int first = (blockIdx.y * kWaves + wave) * per_wave, step = gridDim.y * kWaves * per_wave;

  // A lane's unit of the heads at h0: its head's kind, the element offsets of the unit's two runs of
  // four, and what is read.  A unit's elements are in flight while the one before it is done, and the
  // first one's while the sines are formed.
  struct Unit {
    int head, kvh, e0, e1;
    bool is_q, is_v, turn;
    u32x2 x0, x1;
  };
  const uint16_t* const q_row = p.q + (int64_t)token * p.ldq;
  const uint16_t* const k_row = p.k + (int64_t)token * p.ldk;
  const uint16_t* const v_row = p.v + (int64_t)token * p.ldv;
  uint16_t* const q_out = p.q_out + (int64_t)token * p.ldqo;
  const auto unit_of = [&](int h0, const uint16_t* q_row, const uint16_t* k_row, const uint16_t* v_row) {
    Unit u;
    u.head = h0 + (lane >> p.lanes_log2);
    u.is_q = u.head < p.q_heads;
    u.is_v = u.head >= p.q_heads + p.kv_heads;
    u.kvh = u.is_v ? u.head - p.q_heads - p.kv_heads : u.head - p.q_heads;
    u.turn = !u.is_v && e < turned;
    u.e0 = 8 * e;
    u.e1 = 8 * e + 4;
    if (u.turn && !INTERLEAVED) {
      u.e0 = 4 * e;
      u.e1 = p.half + 4 * e;
    }
    u.x0 = u.x1 = u32x2{0u, 0u};
    if (u.head < heads && e < per_head) {
      const uint16_t* src = (u.is_v ? v_row : u.is_q ? q_row : k_row) +
                            __mul24(u.is_q ? u.head : u.kvh, p.d);
      u.x0 = *reinterpret_cast<const u32x2*>(src + u.e0);
      u.x1 = *reinterpret_cast<const u32x2*>(src + u.e1);
    }
    return u;
  };
  Unit next = unit_of(first, q_row, k_row, v_row);
  const int64_t slot = p.slots[token];

  if (tid < p.half) {
    int axis = 0;
    while (axis + 1 < p.axes && tid >= p.end[axis]) ++axis;
    const double angle =
        (double)p.positions[(long)axis * p.tokens + token] * (double)p.inv_freq[tid];
    const double turns = angle * 0.15915494309189533577;  // 1 / (2 pi)
    sincospif(2.f * (float)(turns - rint(turns)), &sn[tid], &cs[tid]);
  }
  const bool real = slot >= 0 && slot < p.total_slots;
  const int64_t page = real ? page_of(slot, p.page_size, p.total_slots) : 0;
  const int64_t in_page = real ? slot - page * p.page_size : 0;
  const int64_t cache_at = page * p.page_stride + in_page * p.slot_stride;
  const int64_t pair_at = page * p.pair_page + in_page * p.pair_slot;
  __syncthreads();

  for (int h0 = first; h0 < heads; h0 += step) {
    const Unit u = next;
    if (h0 + step < heads) next = unit_of(h0 + step, q_row, k_row, v_row);
    const int head = u.head, kvh = u.kvh, e0 = u.e0, e1 = u.e1;
    const bool is_q = u.is_q, is_v = u.is_v, turn = u.turn;
    const bool in = head < heads && e < per_head && (is_q || real);
    const uint16_t* weight = is_q ? p.q_norm : is_v ? nullptr : p.k_norm;
    u32x2 w0 = {0u, 0u}, w1 = {0u, 0u};
    if (in && weight != nullptr) {
      w0 = *reinterpret_cast<const u32x2*>(weight + e0);
      w1 = *reinterpret_cast<const u32x2*>(weight + e1);
    }
    float a[4], b[4];
    unpack4<BF16>(u.x0, a);
    unpack4<BF16>(u.x1, b);
    if (p.q_norm != nullptr || p.k_norm != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = __builtin_fmaf(a[i], a[i], __builtin_fmaf(b[i], b[i], ss));
      ss = lanes_sum(ss, lanes);
      if (weight != nullptr) {
        const float r = rsqrtf(__builtin_fmaf(ss, p.inv_d, p.eps));
        float wa[4], wb[4];
        unpack4<BF16>(w0, wa);
        unpack4<BF16>(w1, wb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] *= r * wa[i];
          b[i] *= r * wb[i];
        }
      }
    }
    if (turn) {
      const f32x4 c = *reinterpret_cast<const f32x4*>(cs + 4 * e);
      const f32x4 s = *reinterpret_cast<const f32x4*>(sn + 4 * e);
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x0 = a[2 * i], y0 = a[2 * i + 1], x1 = b[2 * i], y1 = b[2 * i + 1];
          a[2 * i] = x0 * c[i] - y0 * s[i];
          a[2 * i + 1] = y0 * c[i] + x0 * s[i];
          b[2 * i] = x1 * c[i + 2] - y1 * s[i + 2];
          b[2 * i + 1] = y1 * c[i + 2] + x1 * s[i + 2];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x0 = a[i], y0 = b[i];
          a[i] = x0 * c[i] - y0 * s[i];
          b[i] = y0 * c[i] + x0 * s[i];
        }
      }
    }
    if (in && is_q) {
      uint16_t* dst = q_out + __mul24(head, p.d);
      *reinterpret_cast<u32x2*>(dst + e0) = pack4<BF16>(a);
      *reinterpret_cast<u32x2*>(dst + e1) = pack4<BF16>(b);
    }
    if constexpr (CACHE == kCache4) {
      if (h0 + per_wave <= p.q_heads || !real) continue;  // (the wave's heads are all q's)
      float* const row = rows[wave] + (lane - e) * 8;
      *reinterpret_cast<f32x4*>(row + (e < per_head ? e0 : 8 * e)) = f32x4{a[0], a[1], a[2], a[3]};
      *reinterpret_cast<f32x4*>(row + (e < per_head ? e1 : 8 * e + 4)) =
          f32x4{b[0], b[1], b[2], b[3]};
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      float x[8];
      *reinterpret_cast<f32x4*>(x) = *reinterpret_cast<const f32x4*>(row + 8 * e);
      *reinterpret_cast<f32x4*>(x + 4) = *reinterpret_cast<const f32x4*>(row + 8 * e + 4);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      uint32_t pair;
      const int per_group = p.group / 8;
      const uint32_t codes = quantize8<BF16>(x, in, p.group < p.d ? per_group : lanes, pair);
      if (in && !is_q) {
        uint8_t* base = static_cast<uint8_t*>(is_v ? p.vc : p.kc);
        const int64_t at = cache_at + kvh * p.head_stride + 8 * e;
        *reinterpret_cast<uint32_t*>(base + at / 2) = codes;
        if (e % per_group == 0)
          (is_v ? p.v_pairs : p.k_pairs)[pair_at + kvh * p.pair_head + e / per_group] = pair;
      }
    } else if (in && !is_q) {
      const int64_t at = cache_at + kvh * p.head_stride;
      if constexpr (CACHE == kCacheE4m3) {
        uint8_t* base = static_cast<uint8_t*>(is_v ? p.vc : p.kc);
        const float* sc = is_v ? p.v_scale : p.k_scale;
        const float scale = sc != nullptr ? sc[kvh] : 1.f;
        *reinterpret_cast<uint32_t*>(base + at + e0) = pack4_e4m3(a, scale);
        *reinterpret_cast<uint32_t*>(base + at + e1) = pack4_e4m3(b, scale);
      } else {
        uint16_t* base = static_cast<uint16_t*>(is_v ? p.vc : p.kc);
        *reinterpret_cast<u32x2*>(base + at + e0) = pack4<BF16>(a);
        *reinterpret_cast<u32x2*>(base + at + e1) = pack4<BF16>(b);
      }
    }
  }
}

struct ReadArgs {
  const uint8_t *kc, *vc;
  const uint32_t *k_pairs, *v_pairs;
  const int64_t* slots;
  uint16_t *k_out, *v_out;
  int64_t page_stride, slot_stride, head_stride;
  int64_t pair_page, pair_slot, pair_head;
  int64_t total_slots;
  int kv_heads, d, page_size, group, ldk, ldv;
};

// A work-group a token, a thread eight elements at a time.  Bound by memory and the launch.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void cache4_read_kernel(ReadArgs p) {
  using A = Act<BF16>;
  const int64_t token = blockIdx.x, slot = p.slots[token];
  const bool real = slot >= 0 && slot < p.total_slots;
  const int64_t page = real ? page_of(slot, p.page_size, p.total_slots) : 0;
  const int64_t in_page = real ? slot - page * p.page_size : 0;
  const int per_head = p.d / 8, units = p.kv_heads * per_head;
  for (int u = threadIdx.x; u < 2 * units; u += kThreads) {
    const bool is_v = u >= units;
    uint16_t* out = is_v ? p.v_out : p.k_out;
    if (out == nullptr) continue;
    const int head = (is_v ? u - units : u) / per_head, e = (is_v ? u - units : u) % per_head;
    u32x4 w = {0u, 0u, 0u, 0u};
    if (real) {
      const int64_t at = page * p.page_stride + in_page * p.slot_stride + head * p.head_stride;
      const int64_t pair_at = page * p.pair_page + in_page * p.pair_slot + head * p.pair_head;
      const uint32_t codes =
          *reinterpret_cast<const uint32_t*>((is_v ? p.vc : p.kc) + at / 2 + 4 * e);
      const uint32_t pair = (is_v ? p.v_pairs : p.k_pairs)[pair_at + 8 * e / p.group];
      const float scale = A::value((uint16_t)pair), offset = A::value((uint16_t)(pair >> 16));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = __builtin_fmaf(scale, (float)(codes >> (8 * i) & 15), offset);
        const float y = __builtin_fmaf(scale, (float)(codes >> (8 * i + 4) & 15), offset);
        w[i] = (uint32_t)A::round(x) | (uint32_t)A::round(y) << 16;
      }
    }
    *reinterpret_cast<u32x4*>(out + token * (is_v ? p.ldv : p.ldk) + (int64_t)head * p.d + 8 * e) =
        w;
  }
}

}  // namespace

hipError_t launch_norm_rope_append(const wq_norm_rope_args& a, hipStream_t stream) {
  AppendArgs p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.k = static_cast<const uint16_t*>(a.k);
  p.v = static_cast<const uint16_t*>(a.v);
  p.q_norm = a.q_heads > 0 ? static_cast<const uint16_t*>(a.q_norm) : nullptr;
  p.k_norm = static_cast<const uint16_t*>(a.k_norm);
  p.q_out = static_cast<uint16_t*>(a.q_out);
  p.kc = a.cache.k;
  p.vc = a.cache.v;
  p.k_pairs = static_cast<uint32_t*>(a.pairs.k);
  p.v_pairs = static_cast<uint32_t*>(a.pairs.v);
  p.k_scale = a.cache.k_scale;
  p.v_scale = a.cache.v_scale;
  p.slots = a.slots;
  p.positions = a.positions;
  p.inv_freq = a.inv_freq;
  p.page_stride = a.cache.page_stride;
  p.slot_stride = a.cache.slot_stride;
  p.head_stride = a.cache.head_stride;
  p.pair_page = a.pairs.page_stride;
  p.pair_slot = a.pairs.slot_stride;
  p.pair_head = a.pairs.head_stride;
  p.total_slots = (int64_t)a.cache.num_pages * a.cache.page_size;
  p.tokens = a.tokens;
  p.q_heads = a.q_heads;
  p.kv_heads = a.cache.kv_heads;
  p.d = a.cache.head_dim;
  p.half = a.rot_dim / 2;
  p.page_size = a.cache.page_size;
  p.group = a.pairs.group_size;
  p.ldq = a.ldq;
  p.ldk = a.ldk;
  p.ldv = a.ldv;
  p.ldqo = a.ldqo;
  p.axes = a.axes;
  p.eps = a.eps;
  p.inv_d = 1.f / (float)p.d;
  int end = 0;
  for (int i = 0; i < a.axes; ++i) p.end[i] = end += a.sections[i];
  while (8 << p.lanes_log2 < p.d) ++p.lanes_log2;
  const int heads = p.q_heads + 2 * p.kv_heads;
  const int per_group = kWaves * (64 >> p.lanes_log2);  // heads a work-group takes at a time
  // Few tokens: a head for each set of lanes.  Many: a work-group forms its token's sines and
  // cosines for several heads (us with one and two work-groups a token, and as many as have heads,
  // 48 heads of 128, 4-bit, with the read: 1 token 6.4, 5.9, 5.7; 256 9.1, 8.5, 8.1; 512 10.0, 9.5, 9.8;
  // 1024 14.9, 15.6, 16.5; 2048 23.2, 23.2, 25.6.  27 heads of 80, E4M3: 256 4.5, 3.9, 3.9; 1024 6.5, 6.2,
  // 6.2; 2048 8.9, 10.4, 10.4).
  const int all = (heads + per_group - 1) / per_group;
  const int parts = a.tokens <= 256 ? all : a.tokens <= 1024 ? std::min(all, 2) : 1;
  const dim3 grid((unsigned)a.tokens, (unsigned)parts);
  const bool bf16 = (a.flags & WQ_FLAG_BF16) != 0;
  const int cache = (a.flags & WQ_FLAG_KV4) ? kCache4 : (a.flags & WQ_FLAG_FP8) ? kCacheE4m3 : kCache16;
#define WQ_APPEND(B, C)                                                                        \
  if (a.interleaved)                                                                           \
    hipLaunchKernelGGL((norm_rope_append_kernel<B, C, true>), grid, dim3(kThreads), 0, stream, p); \
  else                                                                                         \
    hipLaunchKernelGGL((norm_rope_append_kernel<B, C, false>), grid, dim3(kThreads), 0, stream, p)
#define WQ_APPEND_CACHE(B)                    \
  if (cache == kCache4) {                     \
    WQ_APPEND(B, kCache4);                    \
  } else if (cache == kCacheE4m3) {           \
    WQ_APPEND(B, kCacheE4m3);                 \
  } else {                                    \
    WQ_APPEND(B, kCache16);                   \
  }
  if (bf16) {
    WQ_APPEND_CACHE(true)
  } else {
    WQ_APPEND_CACHE(false)
  }
#undef WQ_APPEND_CACHE
#undef WQ_APPEND
  return hipGetLastError();
}

hipError_t launch_cache4_read(const wq_cache4_read_args& a, hipStream_t stream) {
  ReadArgs p{};
  p.kc = static_cast<const uint8_t*>(a.cache.k);
  p.vc = static_cast<const uint8_t*>(a.cache.v);
  p.k_pairs = static_cast<const uint32_t*>(a.pairs.k);
  p.v_pairs = static_cast<const uint32_t*>(a.pairs.v);
  p.slots = a.slots;
  p.k_out = static_cast<uint16_t*>(a.k_out);
  p.v_out = static_cast<uint16_t*>(a.v_out);
  p.page_stride = a.cache.page_stride;
  p.slot_stride = a.cache.slot_stride;
  p.head_stride = a.cache.head_stride;
  p.pair_page = a.pairs.page_stride;
  p.pair_slot = a.pairs.slot_stride;
  p.pair_head = a.pairs.head_stride;
  p.total_slots = (int64_t)a.cache.num_pages * a.cache.page_size;
  p.kv_heads = a.cache.kv_heads;
  p.d = a.cache.head_dim;
  p.page_size = a.cache.page_size;
  p.group = a.pairs.group_size;
  p.ldk = a.ldk;
  p.ldv = a.ldv;
  const dim3 grid((unsigned)a.tokens);
  if (a.flags & WQ_FLAG_BF16)
    hipLaunchKernelGGL((cache4_read_kernel<true>), grid, dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((cache4_read_kernel<false>), grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace wq
