// Rotary positions and the paged cache write of new tokens (wq_rope_append).
//
// Pair i of every q and k head turns by angle position[axis(i)] * inv_freq[i].  The angle is
// formed and reduced by whole turns in fp64 (a position of 10^6 times an fp32 frequency loses
// the phase in fp32), the sine and cosine of what is left are fp32.  A work-group handles
// some of the units of one token: it forms the token's sines and cosines once, in LDS, and
// its threads then each move one unit of 8 elements at a time.
//
// Every element is read once and written once, so many tokens are bound by memory (2048 tokens of
// 32 + 2 x 8 heads of 128 into an E4M3 cache: 11.4 us, 4.0 TB/s) and few by the launch and the
// trips to memory for the position and the rows (one token: 3.1 us).
#include <algorithm>

#include "wq_decode.h"
#include "wq_device.h"

namespace wq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;  // head_dim <= 256

struct RopeArgs {
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  void *kc, *vc;
  const float *k_scale, *v_scale;
  const int64_t* slots;
  const int32_t* positions;
  const float* inv_freq;
  int64_t page_stride, slot_stride, head_stride, total_slots;
  int tokens, q_heads, kv_heads, d, half, page_size;
  int ldq, ldk, ldv, ldqo;
  int end[WQ_MAX_ROPE_AXES];  // first pair past each axis
  int axes;
};

// Four 16-bit values, two dwords.
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

// Stores 4 elements at element offset `at` of a 16-bit tensor or an E4M3 cache.
template <bool BF16, bool FP8>
__device__ __forceinline__ void store4(void* base, int64_t at, const float* f, float scale) {
  if constexpr (FP8)
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(base) + at) = pack4_e4m3(f, scale);
  else
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(base) + at) = pack4<BF16>(f);
}

template <bool BF16, bool FP8, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(RopeArgs p) {
  __shared__ __align__(16) float cs[kMaxPairs], sn[kMaxPairs];
  const int token = blockIdx.x;
  const int tid = threadIdx.x;
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
  const int64_t cache_at =
      page * p.page_stride + (real ? slot - page * p.page_size : 0) * p.slot_stride;
  __syncthreads();

  // Units of a token: per q and k head, rot/8 rotated units of four pairs and (d - rot)/8
  // copied ones, then d/8 units per v head.
  const int rot = 2 * p.half;
  const int per_head = p.d / 8;
  const int turned = rot / 8;
  const int qk = (p.q_heads + p.kv_heads) * per_head;
  const int units = qk + p.kv_heads * per_head;
  for (int u = blockIdx.y * kThreads + tid; u < units; u += gridDim.y * kThreads) {
    const int head = u / per_head, e = u - head * per_head;
    const bool is_v = u >= qk, is_q = head < p.q_heads;
    const int kvh = is_v ? head - p.q_heads - p.kv_heads : head - p.q_heads;
    if (!is_q && !real) continue;
    const uint16_t* src = is_v   ? p.v + (int64_t)token * p.ldv + (int64_t)kvh * p.d
                          : is_q ? p.q + (int64_t)token * p.ldq + (int64_t)head * p.d
                                 : p.k + (int64_t)token * p.ldk + (int64_t)kvh * p.d;
    // element offsets of the unit's two runs of four
    int e0 = 8 * e, e1 = 8 * e + 4;
    const bool turn = !is_v && e < turned;
    if (turn && !INTERLEAVED) {
      e0 = 4 * e;
      e1 = p.half + 4 * e;
    }
    float a[4], b[4];
    unpack4<BF16>(*reinterpret_cast<const u32x2*>(src + e0), a);
    unpack4<BF16>(*reinterpret_cast<const u32x2*>(src + e1), b);
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
    if (is_q) {
      const int64_t at = (int64_t)token * p.ldqo + (int64_t)head * p.d;
      store4<BF16, false>(p.q_out, at + e0, a, 1.f);
      store4<BF16, false>(p.q_out, at + e1, b, 1.f);
    } else {
      const int64_t at = cache_at + kvh * p.head_stride;
      float scale = 1.f;
      if constexpr (FP8) {
        const float* sc = is_v ? p.v_scale : p.k_scale;
        if (sc != nullptr) scale = sc[kvh];
      }
      void* base = is_v ? p.vc : p.kc;
      store4<BF16, FP8>(base, at + e0, a, scale);
      store4<BF16, FP8>(base, at + e1, b, scale);
    }
  }
}

}  // namespace

hipError_t launch_rope_append(const wq_rope_args& a, hipStream_t stream) {
  RopeArgs p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.k = static_cast<const uint16_t*>(a.k);
  p.v = static_cast<const uint16_t*>(a.v);
  p.q_out = static_cast<uint16_t*>(a.q_out);
  p.kc = a.cache.k;
  p.vc = a.cache.v;
  p.k_scale = a.cache.k_scale;
  p.v_scale = a.cache.v_scale;
  p.slots = a.slots;
  p.positions = a.positions;
  p.inv_freq = a.inv_freq;
  p.page_stride = a.cache.page_stride;
  p.slot_stride = a.cache.slot_stride;
  p.head_stride = a.cache.head_stride;
  p.total_slots = (int64_t)a.cache.num_pages * a.cache.page_size;
  p.tokens = a.tokens;
  p.q_heads = a.q_heads;
  p.kv_heads = a.cache.kv_heads;
  p.d = a.cache.head_dim;
  p.half = a.rot_dim / 2;
  p.page_size = a.cache.page_size;
  p.ldq = a.ldq;
  p.ldk = a.ldk;
  p.ldv = a.ldv;
  p.ldqo = a.ldqo;
  p.axes = a.axes;
  int end = 0;
  for (int i = 0; i < a.axes; ++i) p.end[i] = end += a.sections[i];
  const int units = (p.q_heads + 2 * p.kv_heads) * (p.d / 8);
  // Few tokens: a unit per thread.  Many: a work-group forms its token's sines and cosines for
  // several units a thread (us with one, two and three work-groups a token, 768 units, E4M3:
  // 1 token 4.12, 3.78, 3.38; 256 4.68, 4.36, 4.26; 512 5.67, 5.01, 5.45; 1024 7.99, 7.63, 9.04;
  // 2048 11.2, 12.1, 13.5).
  const int all = (units + kThreads - 1) / kThreads;
  const int parts = a.tokens <= 256 ? all : a.tokens <= 1024 ? std::min(all, 2) : 1;
  const dim3 grid((unsigned)a.tokens, (unsigned)parts);
  const bool bf16 = (a.flags & WQ_FLAG_BF16) != 0, fp8 = (a.flags & WQ_FLAG_FP8) != 0;
#define WQ_ROPE(B, F, I)                                                                     \
  hipLaunchKernelGGL((rope_append_kernel<B, F, I>), grid, dim3(kThreads), 0, stream, p)
#define WQ_ROPE_F(B, F)                                                                      \
  if (a.interleaved) WQ_ROPE(B, F, true);                                                    \
  else WQ_ROPE(B, F, false)
  if (bf16) {
    if (fp8) { WQ_ROPE_F(true, true); } else { WQ_ROPE_F(true, false); }
  } else {
    if (fp8) { WQ_ROPE_F(false, true); } else { WQ_ROPE_F(false, false); }
  }
#undef WQ_ROPE_F
#undef WQ_ROPE
  return hipGetLastError();
}

}  // namespace wq
