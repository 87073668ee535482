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
#include <algorithm>

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
  float eps;
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

// Eight elements of a group whose lanes are `width` wide: their codes, and the group's pair.  A
// lane past the head's end takes part with `in` false.
template <bool BF16>
__device__ __forceinline__ uint32_t quantize8(const float* x, bool in, int width, uint32_t& pair) {
  using A = Act<BF16>;
  float low = INFINITY, high = -INFINITY, bad = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    low = fminf(low, in ? x[i] : INFINITY);
    high = fmaxf(high, in ? x[i] : -INFINITY);
    bad += in ? x[i] * 0.f : 0.f;  // NaN for a NaN or an infinity
  }
  for (int w = 1; w < width; w *= 2) {
    low = fminf(low, __shfl_xor(low, w));
    high = fmaxf(high, __shfl_xor(high, w));
    bad += __shfl_xor(bad, w);
  }
  uint32_t sbits = A::round((high - low) / 15.f), obits = A::round(low);
  float scale = A::value((uint16_t)sbits);
  const float offset = A::value((uint16_t)obits);
  if (!((scale - scale) + (offset - offset) + bad == 0.f)) {
    sbits = obits = A::round(__builtin_nanf(""));
    scale = 0.f;
  }
  pair = sbits | obits << 16;
  uint32_t codes = 0;
  if (scale > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = fminf(fmaxf(rintf((x[i] - offset) / scale), 0.f), 15.f);
      codes |= (uint32_t)c << (4 * i);
    }
  }
  return codes;
}

template <bool BF16, int CACHE, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void norm_rope_append_kernel(AppendArgs p) {
  __shared__ __align__(16) float cs[kMaxPairs], sn[kMaxPairs];
  __shared__ __align__(16) float rows[CACHE == kCache4 ? kWaves : 1][64 * 8];
  const int token = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid < p.half) {
    int axis = 0;
    while (axis + 1 < p.axes && tid >= p.end[axis]) ++axis;
    const double angle =
        (double)p.positions[(long)axis * p.tokens + token] * (double)p.inv_freq[tid];
    const double turns = angle * 0.15915494309189533577;  // 1 / (2 pi)
    sincospif(2.f * (float)(turns - rint(turns)), &sn[tid], &cs[tid]);
  }
  const int64_t slot = p.slots[token];
  const bool real = slot >= 0 && slot < p.total_slots;
  const int64_t page = real ? slot / p.page_size : 0;
  const int64_t in_page = real ? slot - page * p.page_size : 0;
  const int64_t cache_at = page * p.page_stride + in_page * p.slot_stride;
  const int64_t pair_at = page * p.pair_page + in_page * p.pair_slot;
  __syncthreads();

  const int lanes = 1 << p.lanes_log2, per_wave = 64 >> p.lanes_log2;
  const int e = lane & (lanes - 1);
  const int per_head = p.d / 8, turned = p.half / 4;  // units of eight elements; turned ones
  const int heads = p.q_heads + 2 * p.kv_heads;
  const int first = (blockIdx.y * kWaves + wave) * per_wave, step = gridDim.y * kWaves * per_wave;
  for (int h0 = first; h0 < heads; h0 += step) {
    const int head = h0 + (lane >> p.lanes_log2);
    const bool is_q = head < p.q_heads, is_v = head >= p.q_heads + p.kv_heads;
    const bool in = head < heads && e < per_head && (is_q || real);
    const int kvh = is_v ? head - p.q_heads - p.kv_heads : head - p.q_heads;
    // element offsets of the unit's two runs of four
    const bool turn = !is_v && e < turned;
    int e0 = 8 * e, e1 = 8 * e + 4;
    if (turn && !INTERLEAVED) {
      e0 = 4 * e;
      e1 = p.half + 4 * e;
    }
    float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
    const uint16_t* weight = is_q ? p.q_norm : is_v ? nullptr : p.k_norm;
    u32x2 w0 = {0u, 0u}, w1 = {0u, 0u};
    if (in) {
      const uint16_t* src = is_v   ? p.v + (int64_t)token * p.ldv + (int64_t)kvh * p.d
                            : is_q ? p.q + (int64_t)token * p.ldq + (int64_t)head * p.d
                                   : p.k + (int64_t)token * p.ldk + (int64_t)kvh * p.d;
      const u32x2 x0 = *reinterpret_cast<const u32x2*>(src + e0);
      const u32x2 x1 = *reinterpret_cast<const u32x2*>(src + e1);
      if (weight != nullptr) {
        w0 = *reinterpret_cast<const u32x2*>(weight + e0);
        w1 = *reinterpret_cast<const u32x2*>(weight + e1);
      }
      unpack4<BF16>(x0, a);
      unpack4<BF16>(x1, b);
    }
    if (p.q_norm != nullptr || p.k_norm != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = __builtin_fmaf(a[i], a[i], __builtin_fmaf(b[i], b[i], ss));
      for (int w = 1; w < lanes; w *= 2) ss += __shfl_xor(ss, w);
      if (weight != nullptr) {
        const float r = 1.f / sqrtf(ss / (float)p.d + p.eps);
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
      uint16_t* dst = p.q_out + (int64_t)token * p.ldqo + (int64_t)head * p.d;
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

// A work-group a token, a thread eight elements at a time.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void cache4_read_kernel(ReadArgs p) {
  using A = Act<BF16>;
  const int64_t token = blockIdx.x, slot = p.slots[token];
  const bool real = slot >= 0 && slot < p.total_slots;
  const int64_t page = real ? slot / p.page_size : 0;
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
  int end = 0;
  for (int i = 0; i < a.axes; ++i) p.end[i] = end += a.sections[i];
  while (8 << p.lanes_log2 < p.d) ++p.lanes_log2;
  const int heads = p.q_heads + 2 * p.kv_heads;
  const int per_group = kWaves * (64 >> p.lanes_log2);  // heads a work-group takes at a time
  // Few tokens: a head for each set of lanes.  Many: a work-group forms its token's sines and
  // cosines for several heads.
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
