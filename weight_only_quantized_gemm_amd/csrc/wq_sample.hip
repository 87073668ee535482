// The next token of each row of logits (wq_sample).
//
// Which tokens stay is a cut in the order of the logits, equal ones by number: the k-th token
// (top_k), or the one at which the sum of p = exp((z - max) / T) passes top_p of the sum (top_p).
// The cut is a pair (key, index), the key a logit's bits made to ascend with its value.  The token
// is then where the sum of what stays, in order of numbers, passes u times the whole.
//
// Borders decide, so p is formed in fp64 (of the logits' exact difference, to some 1e-14) and
// summed as integers, in steps of 2^-44: the sums are the same in any order.
#include "wq_decode.h"
#include "wq_device.h"

namespace wq {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
typedef unsigned long long u64;

enum LogitType { kFp16, kBf16, kFp32 };

struct SampleArgs {
  const void* logits;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* ids;
  float* logprob;
  int64_t ld;
  int vocab;
};

// Ascends with the value; -0 is 0.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __builtin_bit_cast(float, key >> 31 ? key & 0x7fffffffu : ~key);
}

// 2^t for t <= 0, to 2^-52 of its value: the power series of 2^r about 0 up to its twelfth power,
// whose next term is below 2^-53 for |r| <= 1/2.
__device__ __forceinline__ double exp2_neg(double t) {
  if (!(t > -1000.)) return 0.;
  const double n = rint(t), r = t - n;
  double x = 2.5678435993488196e-11;   // ln(2)^12 / 12!
  x = fma(x, r, 4.44553827187081e-10);
  x = fma(x, r, 7.054911620801121e-09);
  x = fma(x, r, 1.0178086009239696e-07);
  x = fma(x, r, 1.3215486790144305e-06);
  x = fma(x, r, 1.5252733804059838e-05);
  x = fma(x, r, 0.00015403530393381606);
  x = fma(x, r, 0.0013333558146428441);
  x = fma(x, r, 0.009618129107628477);
  x = fma(x, r, 0.055504108664821576);
  x = fma(x, r, 0.2402265069591007);
  x = fma(x, r, 0.6931471805599453);
  x = fma(x, r, 1.);
  return __builtin_ldexp(x, (int)n);
}

// The row's probabilities: exponent of p in base 2, p, and p in steps of 2^-44.
struct Weights {
  double top, rate;  // the largest logit; log2(e) / T
  __device__ double exponent(float z) const {
    return (double)z == top ? 0. : ((double)z - top) * rate;
  }
  __device__ double p(float z) const { return z == -INFINITY ? 0. : exp2_neg(exponent(z)); }
  __device__ static u64 steps(double p) {
    // the integer nearest to 2^44 p lies in the low bits of its sum with 2^52
    return __builtin_bit_cast(u64, fma(p, 0x1p44, 0x1p52)) & ((1ull << 52) - 1);
  }
};

// A row as 16-byte vectors that are aligned in memory, whatever its first element is: vector i
// holds elements i * kLen - skew and on; what lies outside the row is not read.
template <int TYPE>
struct Row {
  static constexpr int kLen = TYPE == kFp32 ? 4 : 8;
  static constexpr int kChunk = 64 * kLen;  // elements that a wave takes at a time
  const char* base;
  int vocab, skew, chunks;

  __device__ Row(const SampleArgs& p, int row) {
    constexpr int kSize = 16 / kLen;
    const char* first = static_cast<const char*>(p.logits) + row * p.ld * kSize;
    skew = (int)((uintptr_t)first % 16) / kSize;
    base = first - skew * kSize;
    vocab = p.vocab;
    chunks = (vocab + skew + kChunk - 1) / kChunk;
  }
  // The number of a lane's first element of a chunk.
  __device__ int first(int chunk, int lane) const { return (chunk * 64 + lane) * kLen - skew; }
  __device__ void load(int chunk, int lane, float* z) const {
    const int at = first(chunk, lane);
    const char* src = base + ((int64_t)chunk * 64 + lane) * 16;
    u32x4 w = {0u, 0u, 0u, 0u};
    if (at >= 0 && at + kLen <= vocab) {
      w = *reinterpret_cast<const u32x4*>(src);
    } else if constexpr (TYPE == kFp32) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i >= 0 && at + i < vocab) w[i] = reinterpret_cast<const uint32_t*>(src)[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i >= 0 && at + i < vocab)
          w[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(src)[i] << (16 * (i % 2));
    }
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      const uint32_t bits = w[TYPE == kFp32 ? i : i / 2];
      if constexpr (TYPE == kFp32)
        z[i] = __builtin_bit_cast(float, bits);
      else
        z[i] = Act<TYPE == kBf16>::value((uint16_t)(bits >> (16 * (i % 2))));
    }
  }
  __device__ bool has(int at) const { return at >= 0 && at < vocab; }
};

__device__ __forceinline__ u64 wave_sum(u64 x) {
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) x += __shfl_xor(x, d);
  return x;
}

// The last token that stays: those of a larger key stay, and those of this key up to the index.
struct Cut {
  uint32_t key;
  int index;
  __device__ bool keeps(uint32_t k, int at) const { return k > key || (k == key && at <= index); }
};

constexpr int kMaxChunks = WQ_SAMPLE_MAX_VOCAB / 256 + 1;

struct Shared {
  u64 mass[kMaxChunks];   // of chunks; and of keys' bytes while a cut is sought
  uint32_t count[kMaxChunks];
  uint32_t best_key[kWaves];
  int best_at[kWaves], nan[kWaves];
  // found by one thread for all
  uint32_t key;
  int chunk, index;
  u64 above, total;
  uint32_t above_count;
};

// Exclusive prefix of x[0, n) in place by the first wave; the sum is returned to its lanes.
template <class T>
__device__ T wave_prefix(T* x, int n, int lane) {
  T sum = 0;
  for (int i = 0; i < n; i += 64) {
    const T mine = i + lane < n ? x[i + lane] : 0;
    T upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const T other = __shfl_up(upto, d);
      if (lane >= d) upto += other;
    }
    if (i + lane < n) x[i + lane] = sum + upto - mine;
    sum += __shfl(upto, 63);
  }
  return sum;
}

// One work-group a row.
template <int TYPE>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs p) {
  __shared__ Shared sh;
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Row<TYPE> row(p, r);
  constexpr int kLen = Row<TYPE>::kLen;
  float z[kLen];

  // the largest logit, its first token, and whether there is a NaN
  uint32_t key = 0;
  int at = 0, nan = 0;
  for (int c = wave; c < row.chunks; c += kWaves) {
    row.load(c, lane, z);
    const int first = row.first(c, lane);
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      if (!row.has(first + i)) continue;
      nan |= z[i] != z[i];
      const uint32_t k = key_of(z[i]);
      if (k > key) {
        key = k;
        at = first + i;
      }
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) {
    const uint32_t k = __shfl_xor(key, d);
    const int a = __shfl_xor(at, d);
    nan |= __shfl_xor(nan, d);
    if (k > key || (k == key && a < at)) {
      key = k;
      at = a;
    }
  }
  if (lane == 0) {
    sh.best_key[wave] = key;
    sh.best_at[wave] = at;
    sh.nan[wave] = nan;
  }
  __syncthreads();
  nan = 0;
  key = 0;
  at = 0;
  for (int w = 0; w < kWaves; ++w) {
    nan |= sh.nan[w];
    if (sh.best_key[w] > key || (sh.best_key[w] == key && sh.best_at[w] < at)) {
      key = sh.best_key[w];
      at = sh.best_at[w];
    }
  }
  const float top = value_of(key);
  const float t = p.temperature != nullptr ? p.temperature[r] : 1.f;
  const bool greedy = !(t > 0.f);
  if (nan || top == -INFINITY || greedy) {
    if (tid == 0) {
      const bool bad = nan || top == -INFINITY;
      p.ids[r] = bad ? -1 : at;
      if (p.logprob != nullptr) p.logprob[r] = bad ? __builtin_nanf("") : 0.f;
    }
    return;
  }
  const Weights weights{(double)top, 1.4426950408889634 / (double)t};

  // The cut at which the count of tokens, or the sum of their p, reaches a target: by the bytes of
  // the key from the top, then by number among the tokens of that key.  Leaves in sh.above the sum
  // of p up to the cut.
  const auto find_cut = [&](bool by_count, u64 target) -> Cut {
    uint32_t prefix = 0;
    u64 above = 0;
    uint32_t above_count = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      for (int i = tid; i < 256; i += kThreads) {
        sh.mass[i] = 0;
        sh.count[i] = 0;
      }
      __syncthreads();
      for (int c = wave; c < row.chunks; c += kWaves) {
        row.load(c, lane, z);
        const int first = row.first(c, lane);
#pragma unroll
        for (int i = 0; i < kLen; ++i) {
          const uint32_t k = key_of(z[i]);
          if (!row.has(first + i) || (shift < 24 && (k ^ prefix) >> (shift + 8))) continue;
          atomicAdd(&sh.count[255 - (k >> shift & 255)], 1u);
          atomicAdd(&sh.mass[255 - (k >> shift & 255)], Weights::steps(weights.p(z[i])));
        }
      }
      __syncthreads();
      if (tid == 0) {
        int i = 0;
        for (; i < 255; ++i) {
          if (by_count ? above_count + sh.count[i] >= target : above + sh.mass[i] >= target) break;
          above += sh.mass[i];
          above_count += sh.count[i];
        }
        sh.key = prefix | (uint32_t)(255 - i) << shift;
        sh.above = above;
        sh.above_count = above_count;
      }
      __syncthreads();
      prefix = sh.key;
      above = sh.above;
      above_count = sh.above_count;
    }
    // how many of this key stay
    const u64 each = Weights::steps(weights.p(value_of(prefix)));
    const u64 left = by_count ? target - above_count
                              : (each == 0 ? 1 : (target - above + each - 1) / each);
    __syncthreads();
    for (int c = wave; c < row.chunks; c += kWaves) {
      row.load(c, lane, z);
      const int first = row.first(c, lane);
      int n = 0;
#pragma unroll
      for (int i = 0; i < kLen; ++i) n += row.has(first + i) && key_of(z[i]) == prefix;
#pragma unroll
      for (int d = 32; d >= 1; d /= 2) n += __shfl_xor(n, d);
      if (lane == 0) sh.count[c] = n;
    }
    __syncthreads();
    if (wave == 0) {
      wave_prefix(sh.count, row.chunks, lane);
      if (lane == 0) {
        sh.above = above + left * each;
        sh.index = row.vocab - 1;
      }
      // the chunk in which the left-th of them lies, and it there
      int chunk = 0;
      for (int c = lane; c < row.chunks; c += 64)
        if (sh.count[c] < left) chunk = c;
#pragma unroll
      for (int d = 32; d >= 1; d /= 2) chunk = max(chunk, __shfl_xor(chunk, d));
      row.load(chunk, lane, z);
      const int first = row.first(chunk, lane);
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < kLen; ++i) mine += row.has(first + i) && key_of(z[i]) == prefix;
      uint32_t upto = mine;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const uint32_t other = __shfl_up(upto, d);
        if (lane >= d) upto += other;
      }
      u64 n = sh.count[chunk] + upto - mine;
#pragma unroll
      for (int i = 0; i < kLen; ++i)
        if (row.has(first + i) && key_of(z[i]) == prefix && ++n == left) sh.index = first + i;
    }
    __syncthreads();
    return Cut{prefix, sh.index};
  };

  Cut cut{0, row.vocab};
  const int k = p.top_k != nullptr ? p.top_k[r] : 0;
  const float top_p = p.top_p != nullptr ? p.top_p[r] : 1.f;
  const float min_p = p.min_p != nullptr ? p.min_p[r] : 0.f;
  const bool cut_k = k > 0 && k < row.vocab, cut_p = top_p < 1.f;
  const auto kept = [&](float v, int i) -> double {  // p where the token stays, else 0
    const uint32_t kk = key_of(v);
    if (!row.has(i) || !cut.keeps(kk, i)) return 0.;
    const double x = weights.p(v);
    return kk == key || !(x < (double)min_p) ? x : 0.;
  };
  const auto chunk_sums = [&](bool all) {
    __syncthreads();
    for (int c = wave; c < row.chunks; c += kWaves) {
      row.load(c, lane, z);
      const int first = row.first(c, lane);
      u64 sum = 0;
#pragma unroll
      for (int i = 0; i < kLen; ++i)
        sum += Weights::steps(!all              ? kept(z[i], first + i)
                              : row.has(first + i) ? weights.p(z[i])
                                                   : 0.);
      sum = wave_sum(sum);
      if (lane == 0) sh.mass[c] = sum;
    }
    __syncthreads();
    if (wave == 0) {
      const u64 total = wave_prefix(sh.mass, row.chunks, lane);
      if (lane == 0) sh.total = total;
    }
    __syncthreads();
  };
  u64 total = 0;
  if (cut_k) {
    cut = find_cut(true, (u64)k);
    total = sh.above;
  } else if (cut_p) {
    chunk_sums(true);
    total = sh.total;
  }
  if (cut_p) {
    // the least sum that is not below top_p of the total, and that the first token has at least
    const double want = ceil((double)fmaxf(top_p, 0.f) * (double)total);
    cut = find_cut(false, want < 1. ? 1 : (u64)want);
  }
  chunk_sums(false);
  total = sh.total;

  if (wave == 0) {
    const float u = p.u[r];
    const double want = u > 0.f ? (double)u * (double)total : 0.;
    const u64 pass = want < (double)total ? min((u64)want, total - 1) : total - 1;
    int chunk = 0;
    for (int c = lane; c < row.chunks; c += 64)
      if (sh.mass[c] <= pass) chunk = c;
#pragma unroll
    for (int d = 32; d >= 1; d /= 2) chunk = max(chunk, __shfl_xor(chunk, d));
    row.load(chunk, lane, z);
    const int first = row.first(chunk, lane);
    u64 m[kLen], mine = 0;
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      m[i] = Weights::steps(kept(z[i], first + i));
      mine += m[i];
    }
    u64 upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const u64 other = __shfl_up(upto, d);
      if (lane >= d) upto += other;
    }
    u64 sum = sh.mass[chunk] + upto - mine;
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      const u64 next = sum + m[i];
      if (sum <= pass && pass < next) {
        p.ids[r] = first + i;
        if (p.logprob != nullptr)
          p.logprob[r] = (float)(weights.exponent(z[i]) * 0.6931471805599453 -
                                 log((double)total * 0x1p-44));
      }
      sum = next;
    }
  }
}

}  // namespace

size_t sample_workspace_bytes(int, int, uint32_t) { return 0; }

hipError_t launch_sample(const wq_sample_args& a, hipStream_t stream) {
  SampleArgs p{};
  p.logits = a.logits;
  p.u = a.u;
  p.temperature = a.temperature;
  p.top_k = a.top_k;
  p.top_p = a.top_p;
  p.min_p = a.min_p;
  p.ids = a.ids;
  p.logprob = a.logprob;
  p.ld = a.ld;
  p.vocab = a.vocab;
  const dim3 grid((unsigned)a.rows), block(kThreads);
  if (a.flags & WQ_FLAG_FP32)
    hipLaunchKernelGGL((sample_kernel<kFp32>), grid, block, 0, stream, p);
  else if (a.flags & WQ_FLAG_BF16)
    hipLaunchKernelGGL((sample_kernel<kBf16>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((sample_kernel<kFp16>), grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace wq
