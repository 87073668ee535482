// RMS norm with the residual add: s = x + delta, y = s / sqrt(mean(s^2) + eps) * w.
//
// Two rows read, two written, a few operations per element: bound by memory for many rows
// (bf16, 8192 rows of 8192: 94 us, 5.7 TB/s of the four rows) and by its launch and one trip to
// memory for few (fp16, one row of 4096: 2.7 us).  A row stays in registers as fp32 between its
// one read and its two writes, so nothing is read twice and the norm sees the unrounded sum.
#include "wq_decode.h"
#include "wq_device.h"

namespace wq {
namespace {

// One work-group per row, NPT 16-byte granules (8 elements) per thread.
template <bool BF16, int THREADS, int NPT>
__global__ __launch_bounds__(THREADS) void add_rms_norm_kernel(
    const u32x4* x, const u32x4* delta, const u32x4* w, u32x4* sum_out, u32x4* y, int granules,
    int ldx, int ldd, int lds, int ldy, float inv_n, float eps) {
  using A = Act<BF16>;
  constexpr int WAVES = THREADS / 64;
  __shared__ float red[WAVES];
  const int tid = threadIdx.x;
  const long row = blockIdx.x;
  x += row * (ldx / 8);
  y += row * (ldy / 8);
  if (delta != nullptr) delta += row * (ldd / 8);
  if (sum_out != nullptr) sum_out += row * (lds / 8);

  // every load before any arithmetic (clamped: a granule past the row repeats its last)
  u32x4 xv[NPT], dv[NPT], wv[NPT];
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    const int g = min(tid + i * THREADS, granules - 1);
    xv[i] = x[g];
    if (delta != nullptr) dv[i] = delta[g];
  }
#pragma unroll
  for (int i = 0; i < NPT; ++i) wv[i] = w[min(tid + i * THREADS, granules - 1)];

  float s[NPT][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    const bool real = tid + i * THREADS < granules;
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v = A::value((uint16_t)(xv[i][j / 2] >> (16 * (j % 2))));
      if (delta != nullptr) v += A::value((uint16_t)(dv[i][j / 2] >> (16 * (j % 2))));
      s[i][j] = v;
      part = __builtin_fmaf(v, v, part);
    }
    ss += real ? part : 0.f;
  }
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) ss += __shfl_xor(ss, d);
  if constexpr (WAVES > 1) {
    if ((tid & 63) == 0) red[tid >> 6] = ss;
    __syncthreads();
    ss = red[0];
#pragma unroll
    for (int k = 1; k < WAVES; ++k) ss += red[k];
  }
  const float r = 1.f / sqrtf(ss * inv_n + eps);
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    const int g = tid + i * THREADS;
    if (g >= granules) continue;
    u32x4 yo, so;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float w0 = A::value((uint16_t)wv[i][j]), w1 = A::value((uint16_t)(wv[i][j] >> 16));
      yo[j] = (uint32_t)A::round(s[i][2 * j] * r * w0) |
              ((uint32_t)A::round(s[i][2 * j + 1] * r * w1) << 16);
      so[j] = (uint32_t)A::round(s[i][2 * j]) | ((uint32_t)A::round(s[i][2 * j + 1]) << 16);
    }
    y[g] = yo;
    if (sum_out != nullptr) sum_out[g] = so;
  }
}

template <bool BF16, int THREADS, int NPT>
hipError_t launch_norm_t(const wq_norm_args& a, hipStream_t stream) {
  hipLaunchKernelGGL((add_rms_norm_kernel<BF16, THREADS, NPT>), dim3((unsigned)a.rows),
                     dim3(THREADS), 0, stream, static_cast<const u32x4*>(a.x),
                     static_cast<const u32x4*>(a.delta), static_cast<const u32x4*>(a.weight),
                     static_cast<u32x4*>(a.sum_out), static_cast<u32x4*>(a.y), a.n / 8, a.ldx,
                     a.ldd, a.lds, a.ldy, 1.f / (float)a.n, a.eps);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_norm_type(const wq_norm_args& a, hipStream_t stream) {
  // One granule a thread as far as a work-group goes: a row's loads then leave together (us,
  // one row and 8192 rows, bf16: n 4096, 256 threads of two 2.93 and 48.2, 512 of one 2.69 and
  // 48.5; n 8192, 256 of four 3.50 and 96.2, 1024 of one 3.16 and 91.9; n 32768 and 2048 rows,
  // 256 of sixteen 6.65 and 106.9, 1024 of four 5.49 and 103.8).  A single wave needs no exchange
  // through LDS (n 512: 2.32 and 7.52, 256 threads 2.43 and 9.05), but two granules a thread
  // cost a lone row more than that (n 1024: 2.71 and 2.44).
  const int granules = a.n / 8;
  if (granules <= 64) return launch_norm_t<BF16, 64, 1>(a, stream);
  if (granules <= 256) return launch_norm_t<BF16, 256, 1>(a, stream);
  if (granules <= 512) return launch_norm_t<BF16, 512, 1>(a, stream);
  if (granules <= 1024) return launch_norm_t<BF16, 1024, 1>(a, stream);
  if (granules <= 2048) return launch_norm_t<BF16, 1024, 2>(a, stream);
  if (granules <= 4096) return launch_norm_t<BF16, 1024, 4>(a, stream);
  return launch_norm_t<BF16, 1024, 8>(a, stream);
}

}  // namespace

hipError_t launch_add_rms_norm(const wq_norm_args& a, hipStream_t stream) {
  return (a.flags & WQ_FLAG_BF16) ? launch_norm_type<true>(a, stream)
                                  : launch_norm_type<false>(a, stream);
}

}  // namespace wq
