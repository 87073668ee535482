// The next token of each row of logits (wq_sample).
//
// Which tokens stay is a cut in the order of the logits, equal ones by number: the k-th token
// (top_k), or the one at which the sum of p = exp((z - max) / T) passes top_p of the sum (top_p).
// The cut is a pair (key, index), the key a logit's bits made to ascend with its value.  The token
// is then where the sum of what stays, in order of numbers, passes u times the whole.
//
// Borders decide, so p is formed in fp64 (of the logits' exact difference, to some 4e-14) and
// summed as integers, in steps of 2^-44: the sums are the same in any order.
//
// A row is read three times, by as many work-groups as fill the chip:
//   sample_max     the largest logit of each slice of a row;
//   sample_bins    tokens, and sums of p, by how far a logit lies below the largest, in 2025 bins of
//                  1/45 of a power of two: the cut lies in one of them (top_k and top_p: in one each);
//   sample_gather  the sums of p over what lies above the cut's bin, for each 1 KiB of the row, and a
//                  list of what lies in it;
//   sample_pick    a work-group a row: the list in order, the cut, and the token.
// A bin that holds more tokens than the list is sought again by the bytes of the keys, in passes over
// the row by sample_pick's work-group, five for each cut and one for the sums.  That is slow: 128000
// logits all equal take 1.1 ms with top_p and 2.0 with top_k too, bf16 ones of sd 0.5 around 20, whose
// steps are 0.125, 0.67, fp32 ones of sd 2 at a temperature of 20 0.50 (64 such rows 1.16, 2.1, 0.70 and
// 0.58 ms).  At a temperature of 5 the list holds them (28 us, 64 rows 59).
//
// One row is bound by four launches that need each other's results (128000 logits in bf16: 3.1, 4.0, 4.6
// and 4.8 us), many by the instructions of the fp64 exponentials, 32 a logit (256 such rows: 14.9, 31,
// 28 and 12 us; the first pass runs at 4.4 TB/s).  Without a cut there are three launches, and one of
// them forms p (one row 14 us, 64 24, 256 50; fp32 13 and 27); greedy rows take 9.3 us, 64 14 (fp32 16).
#include <algorithm>
#include <type_traits>

#include "wq_decode.h"
#include "wq_device.h"

namespace wq {
namespace {

typedef unsigned long long u64;
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

enum LogitType { kFp16, kBf16, kFp32 };

constexpr int kThreads = 512, kWaves = kThreads / 64;            // of the kernels on slices
constexpr int kPickThreads = 256, kPickWaves = kPickThreads / 64;  // (a thread a byte value)
constexpr int kMaxSlices = 64;
constexpr int kBins = 2048;  // the last one: p is 0 in steps of 2^-44
constexpr double kBinsPerPower = 45.;
constexpr int kList = 2048;
constexpr int kMaxChunks = WQ_SAMPLE_MAX_VOCAB / 256 + 1;

// Where the cuts lie: the bins of the list, and what is above them.
struct Bins {
  int k, p_low, p_high;  // bin of the k-th token; bins that may hold the token at top_p; -1: no cut
  uint32_t above_k;      // tokens above bin k
  u64 mass_above_k, mass_above_p;  // sums of p above bins k and p_low
  u64 all;                         // and over all of them
  __device__ int first() const { return p_low >= 0 ? p_low : k >= 0 ? k : kBins; }
  __device__ bool lists(int bin) const {
    return bin == k || (bin >= p_low && bin <= p_high && p_low >= 0);
  }
};

struct SampleArgs {
  const void* logits;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* ids;
  float* logprob;
  int64_t ld;
  int vocab, slices, max_chunks;
  // workspace, for each row: [slices], [kBins], [kBins], [max_chunks], [kList], one
  u64* best;        // a slice's largest key and, below it, the first of its tokens, negated
  u64* bin_mass;
  uint32_t* bin_count;
  u64* chunk_mass;
  u64* list;        // keys and negated tokens
  Bins* bins;
  uint32_t* listed;
};

// Ascends with the value; -0 is 0.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __builtin_bit_cast(float, key >> 31 ? key & 0x7fffffffu : ~key);
}

// a * b + c with c in scalar registers: the compiler's own form copies a constant c to vector
// registers each time, because it writes the sum over it.
__device__ __forceinline__ double fma_s(double a, double b, double c) {
  double d;
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "s"(c));
  return d;
}

// x without its fraction, the nearest number of 32 bits where it is none (as the instruction has it,
// and the language does not: infinities are the last, no number and what is below 0 are 0).
__device__ __forceinline__ uint32_t whole_of(double x) {
  uint32_t n;
  asm("v_cvt_u32_f64 %0, %1" : "=v"(n) : "v"(x));
  return n;
}

// 2^t for t <= 0, to 3.7e-14 of its value: 1 + r q(r) for the remainder |r| <= 1/2 of t, q of degree
// 8 through the Chebyshev points.
__device__ __forceinline__ double exp2_neg(double t, int more = 0) {
  t = fmax(t, -1100.);  // (no number too, as -inf less -inf: 0)
  const double n = rint(t), r = t - n;
  double x = fma_s(1.0203121171282166e-07, r, 1.3255224873639605e-06);
  x = fma_s(x, r, 1.5252686845725586e-05);
  x = fma_s(x, r, 1.5403455852474373e-04);
  x = fma_s(x, r, 1.333355817904396e-03);
  x = fma_s(x, r, 9.618129159402536e-03);
  x = fma_s(x, r, 5.550410866476042e-02);
  x = fma_s(x, r, 2.402265069581299e-01);
  x = fma_s(x, r, 6.931471805599453e-01);
  x = fma(x, r, 1.);
  return __builtin_ldexp(x, (int)n + more);
}

// The row's probabilities: exponent of p in base 2, p, p in steps of 2^-44, and the bin.
struct Weights {
  double top, rate;  // the largest logit; log2(e) / T
  __device__ Weights(float largest, float t) : top(largest), rate(1.4426950408889634 / (double)t) {}
  __device__ double exponent(float z) const { return ((double)z - top) * rate; }
  __device__ double p(float z) const { return exp2_neg(exponent(z)); }
  // Steps as a whole number in fp64; of up to 512 tokens they add exactly.
  __device__ static double steps_at(double exponent) { return rint(exp2_neg(exponent, 44)); }
  __device__ static u64 whole(double steps) {
    // the low bits of its sum with 2^52, which rounds what is no whole number
    return __builtin_bit_cast(u64, steps + 0x1p52) & ((1ull << 52) - 1);
  }
  __device__ u64 steps(float z) const { return whole(exp2_neg(exponent(z), 44)); }
  // Never falls as z does.  Below 2^-45 there are no steps.
  __device__ static int bin(double exponent) {
    return (int)min(whole_of(-exponent * kBinsPerPower), (uint32_t)kBins - 1u);
  }
  // A logit below which no token is in a bin before the last, and, with min_p, none stays.
  __device__ float least(float min_p) const {
    constexpr double kDeepest = (kBins - 1) / -kBinsPerPower;
    return logit_below(min_p > 0.f ? fmin(fmax(kDeepest, log2((double)min_p) - 0x1p-10), 0.)
                                   : kDeepest);
  }
  // A logit below which no exponent is above this one.
  __device__ float logit_below(double exponent) const {
    const double z = top + (exponent - 0x1p-20) / rate;
    return (float)(z - fabs(z) * 0x1p-20) - 1e-30f;
  }
};

__device__ __forceinline__ float scalar(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}

// What a row asks for.
struct Setting {
  float t, min_p;
  double top_p;
  int k;
  bool greedy, cut_k, cut_p;

  __device__ Setting(const SampleArgs& p, int row) {
    t = p.temperature != nullptr ? p.temperature[row] : 1.f;
    k = p.top_k != nullptr ? p.top_k[row] : 0;
    float share = p.top_p != nullptr ? p.top_p[row] : 1.f;
    min_p = p.min_p != nullptr ? p.min_p[row] : 0.f;
    t = scalar(t);  // what depends on them is then a branch of the wave
    k = __builtin_amdgcn_readfirstlane(k);
    share = scalar(share);
    min_p = scalar(min_p);
    greedy = !(t > 0.f) || min_p > 1.f;  // (no p is above 1: the first token alone is left)
    cut_k = k > 0 && k < p.vocab;
    cut_p = share < 1.f;
    top_p = share > 0.f ? share : 0.;
  }
  // The least sum that is not below top_p of the total, and that the first token has at least.
  __device__ u64 share_of(u64 total) const {
    const double want = ceil(top_p * (double)total);
    return want < 1. ? 1 : (u64)want;
  }
};

// A row as 16-byte vectors that are aligned in memory, whatever its first element is: vector i
// holds elements i * kLen - skew and on; what lies outside the row is not read.
template <int TYPE>
struct Row {
  static constexpr int kLen = TYPE == kFp32 ? 4 : 8;
  static constexpr int kChunk = 64 * kLen;  // elements that a wave takes at a time
  static constexpr uint32_t kLowest =
      TYPE == kFp32 ? 0xff800000u : TYPE == kBf16 ? 0xff80ff80u : 0xfc00fc00u;  // -inf
  const char* base;
  int vocab, skew, chunks;
  bool infinite = false;  // +inf reads as 0, all others as -inf: they count for nothing beside it

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
  // A lane's vector of a chunk; -inf outside the row.
  __device__ u32x4 raw(int chunk, int lane) const {
    const char* src = base + ((int64_t)chunk * 64 + lane) * 16;
    const int from = first(chunk, 0);
    if (from >= 0 && from + kChunk <= vocab)  // (a condition of the wave's)
      return *reinterpret_cast<const u32x4*>(src);
    const int at = first(chunk, lane);
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = kLowest;
    if (at >= 0 && at + kLen <= vocab) {
      w = *reinterpret_cast<const u32x4*>(src);
    } else if constexpr (TYPE == kFp32) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (has(at + i)) w[i] = reinterpret_cast<const uint32_t*>(src)[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (has(at + i))
          w[i / 2] = (w[i / 2] & (i % 2 ? 0xffffu : 0xffff0000u)) |
                     (uint32_t) reinterpret_cast<const uint16_t*>(src)[i] << (16 * (i % 2));
    }
    return w;
  }
  __device__ static void values(u32x4 w, float* z) {
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      const uint32_t bits = w[TYPE == kFp32 ? i : i / 2];
      if constexpr (TYPE == kFp32)
        z[i] = __builtin_bit_cast(float, bits);
      else
        z[i] = Act<TYPE == kBf16>::value((uint16_t)(bits >> (16 * (i % 2))));
    }
  }
  __device__ void take(u32x4 w, float* z) const {
    values(w, z);
    if (infinite) {
#pragma unroll
      for (int i = 0; i < kLen; ++i) z[i] = z[i] == INFINITY ? 0.f : -INFINITY;
    }
  }
  __device__ void load(int chunk, int lane, float* z) const { take(raw(chunk, lane), z); }
  __device__ bool has(int at) const { return at >= 0 && at < vocab; }
};

// Chunks from + wave, from + wave + waves, ... before `to`, the next one's vector in flight while
// f(chunk, values) runs; `next`: the first one's, requested by first_vector.
template <int TYPE>
__device__ __forceinline__ u32x4 first_vector(const Row<TYPE>& row, int from, int to, int wave,
                                              int lane) {
  return from + wave < to ? row.raw(from + wave, lane) : u32x4{0u, 0u, 0u, 0u};
}
template <int TYPE, class F>
__device__ __forceinline__ void each_chunk(const Row<TYPE>& row, int from, int to, int wave,
                                           int waves, int lane, u32x4 next, F f) {
  for (int c = from + wave; c < to; c += waves) {
    const u32x4 w = next;
    if (c + waves < to) next = row.raw(c + waves, lane);
    float z[Row<TYPE>::kLen];
    row.take(w, z);
    f(c, z);
  }
}

// A step of a scan over the wave's lanes: what lies CTRL before a lane, 0 where nothing does or the
// lane's row is not in ROWS.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t lanes_before(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 lanes_before(u64 x) {
  return lanes_before<CTRL, ROWS>((uint32_t)x) |
         (u64)lanes_before<CTRL, ROWS>((uint32_t)(x >> 32)) << 32;
}
// Inclusive scan: row_shr 1, 2, 4 and 8 within rows of 16 lanes, then a row's last lane to the next
// row, and the first half's last to the second.
template <class T, class F>
__device__ __forceinline__ T wave_scan(T x, F f) {
  x = f(x, lanes_before<0x111, 0xf>(x));
  x = f(x, lanes_before<0x112, 0xf>(x));
  x = f(x, lanes_before<0x114, 0xf>(x));
  x = f(x, lanes_before<0x118, 0xf>(x));
  x = f(x, lanes_before<0x142, 0xa>(x));
  x = f(x, lanes_before<0x143, 0xc>(x));
  return x;
}
template <class T>
__device__ __forceinline__ T wave_upto(T x) {
  return wave_scan(x, [](T a, T b) { return a + b; });
}
__device__ __forceinline__ uint32_t last_lane(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
__device__ __forceinline__ u64 last_lane(u64 x) {
  return last_lane((uint32_t)x) | (u64)last_lane((uint32_t)(x >> 32)) << 32;
}
__device__ __forceinline__ u64 lane_at(u64 x, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)x, lane) |
         (u64)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), lane) << 32;
}
template <class T>
__device__ __forceinline__ T wave_sum(T x) {
  return last_lane(wave_upto(x));
}
template <class T>
__device__ __forceinline__ T wave_max(T x) {
  return last_lane(wave_scan(x, [](T a, T b) { return a > b ? a : b; }));
}

// The slice's chunks.
template <int TYPE>
__device__ __forceinline__ void slice_of(const SampleArgs& p, const Row<TYPE>& row, int slice,
                                         int& from, int& to) {
  from = (int)((int64_t)row.chunks * slice / p.slices);
  to = (int)((int64_t)row.chunks * (slice + 1) / p.slices);
}

constexpr u64 kNan = ~0ull;  // in a slice's best: it holds a NaN

// A token's place in the order: larger keys first, equal ones by number.
__device__ __forceinline__ u64 place_of(uint32_t key, int at) {
  return (u64)key << 32 | (uint32_t)~at;
}
__device__ __forceinline__ uint32_t key_at(u64 place) { return (uint32_t)(place >> 32); }
__device__ __forceinline__ int token_at(u64 place) { return (int)~(uint32_t)place; }

template <int TYPE>
__global__ __launch_bounds__(kThreads) void sample_max(SampleArgs p) {
  __shared__ u64 best_lds[kWaves];
  const int slice = blockIdx.x, r = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Row<TYPE> row(p, r);
  constexpr int kLen = Row<TYPE>::kLen;
  int from, to;
  slice_of(p, row, slice, from, to);
  // The largest value of a lane and the first chunk that has it; the largest bits without signs,
  // by which a NaN shows.
  float top = -INFINITY;
  int top_chunk = from + wave;
  u32x4 sizes = {0u, 0u, 0u, 0u};
  const auto look = [&](int c, u32x4 w) {
    float z[kLen];
    Row<TYPE>::values(w, z);
    float m = fmaxf(z[0], z[1]);
#pragma unroll
    for (int i = 2; i < kLen; ++i) m = fmaxf(m, z[i]);
    if (m > top) {
      top = m;
      top_chunk = c;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kFp32) {
        sizes[i] = max(sizes[i], w[i] & 0x7fffffffu);
      } else {
        const uint32_t a = sizes[i], b = w[i] & 0x7fff7fffu;
        sizes[i] = __builtin_bit_cast(
            uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                __builtin_bit_cast(u16x2, b)));
      }
    }
  };
  int c = from + wave;
  for (; c + 3 * kWaves < to; c += 4 * kWaves) {
    u32x4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = row.raw(c + i * kWaves, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) look(c + i * kWaves, w[i]);
  }
  for (; c < to; c += kWaves) look(c, row.raw(c, lane));
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = sizes[i];
    if constexpr (TYPE == kFp32)
      nan |= x > 0x7f800000u;
    else
      nan |= (x & 0xffffu) > (Row<TYPE>::kLowest & 0x7fffu) ||
             (x >> 16) > (Row<TYPE>::kLowest & 0x7fffu);
  }
  // the first token of the wave's largest value, in one of the lanes that have it
  const uint32_t key = key_of(top), wave_key = wave_max(key);
  u64 best = 0;
  if (from + wave < to && key == wave_key) {
    float z[kLen];
    row.load(top_chunk, lane, z);
#pragma unroll
    for (int i = kLen - 1; i >= 0; --i)
      if (z[i] == top) best = place_of(key, row.first(top_chunk, lane) + i);
  }
  if (nan) best = kNan;
  best = wave_max(best);
  if (lane == 0) best_lds[wave] = best;
  // the row's bins and list start empty
  for (int i = slice * kThreads + tid; i < kBins; i += p.slices * kThreads) {
    p.bin_mass[(int64_t)r * kBins + i] = 0;
    p.bin_count[(int64_t)r * kBins + i] = 0;
  }
  if (slice == 0 && tid == 0) p.listed[r] = 0;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWaves; ++w) best = max(best, best_lds[w]);
    p.best[(int64_t)r * p.slices + slice] = best;
  }
}

// The row's largest logit, as a place, by each wave.
__device__ __forceinline__ u64 row_best(const SampleArgs& p, int r, int lane) {
  return wave_max(lane < p.slices ? p.best[(int64_t)r * p.slices + lane] : 0);
}
__device__ __forceinline__ bool row_is_bad(u64 best) {
  return best == kNan || value_of(key_at(best)) == -INFINITY;
}
// The row's largest logit as Row::take gives it.
template <int TYPE>
__device__ __forceinline__ float row_top(Row<TYPE>& row, u64 best) {
  const float top = value_of(key_at(best));
  row.infinite = top == INFINITY;
  return row.infinite ? 0.f : top;
}

// The largest of a lane's values.
template <int LEN>
__device__ __forceinline__ float largest(const float* z) {
  float m = z[0];
#pragma unroll
  for (int i = 1; i < LEN; ++i) m = fmaxf(m, z[i]);
  return m;
}

// Whether min_p lets a token stay that has this exponent and key.
__device__ __forceinline__ bool min_keeps(double exponent, uint32_t key, uint32_t top_key,
                                          float min_p) {
  return key == top_key || !(exp2_neg(exponent) < (double)min_p);
}

// Rows that are cut: tokens and sums of p by bins.  Others: the sums of their chunks.
template <int TYPE>
__global__ __launch_bounds__(kThreads) void sample_bins(SampleArgs p) {
  __shared__ u64 mass[kBins];
  __shared__ uint32_t count[kBins];
  const int slice = blockIdx.x, r = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Row<TYPE> row(p, r);
  constexpr int kLen = Row<TYPE>::kLen;
  int from, to;
  slice_of(p, row, slice, from, to);
  const u32x4 first = first_vector(row, from, to, wave, lane);
  const Setting set(p, r);
  for (int i = tid; i < kBins; i += kThreads) {
    mass[i] = 0;
    count[i] = 0;
  }
  const u64 best = row_best(p, r, lane);
  if (set.greedy || row_is_bad(best)) return;
  const float top = row_top(row, best);
  const uint32_t top_key = key_of(top);
  const Weights weights(top, set.t);
  if (!(set.cut_k || set.cut_p)) {
    const float least = weights.least(set.min_p);
    each_chunk(row, from, to, wave, kWaves, lane, first, [&](int c, const float* z) {
      double sum = 0.;
      u64 all = 0;
      if (__ballot(largest<kLen>(z) >= least)) {
        if (set.min_p > 0.f) {
#pragma unroll
          for (int i = 0; i < kLen; ++i) {
            const double e = weights.exponent(z[i]);
            if (min_keeps(e, key_of(z[i]), top_key, set.min_p)) sum += Weights::steps_at(e);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kLen; ++i) sum += Weights::steps_at(weights.exponent(z[i]));
        }
        all = wave_sum(Weights::whole(sum));
      }
      if (lane == 0) p.chunk_mass[(int64_t)r * p.max_chunks + c] = all;
    });
    return;
  }
  __syncthreads();
  const float least = weights.least(0.f);
  each_chunk(row, from, to, wave, kWaves, lane, first, [&](int, const float* z) {
    if (!__ballot(largest<kLen>(z) >= least)) return;
    int b[kLen];
    u64 steps[kLen];
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      const double e = weights.exponent(z[i]);
      b[i] = Weights::bin(e);
      if (set.cut_p) steps[i] = Weights::whole(exp2_neg(e, 44));
    }
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      if (b[i] == kBins - 1) continue;
      if (set.cut_k) atomicAdd(&count[b[i]], 1u);
      if (set.cut_p) atomicAdd(&mass[b[i]], steps[i]);
    }
  });
  __syncthreads();
  for (int i = tid; i < kBins - 1; i += kThreads) {
    if (count[i]) atomicAdd(&p.bin_count[(int64_t)r * kBins + i], count[i]);
    if (mass[i]) atomicAdd(&p.bin_mass[(int64_t)r * kBins + i], mass[i]);
  }
}

// A thread's bins of the row, requested before they are known to be needed.
struct MyBins {
  static constexpr int kEach = kBins / kThreads;
  u64 m[kEach];
  uint32_t n[kEach];
  __device__ MyBins(const SampleArgs& p, int r, int tid) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      m[i] = p.bin_mass[(int64_t)r * kBins + kEach * tid + i];
      n[i] = p.bin_count[(int64_t)r * kBins + kEach * tid + i];
    }
  }
};

// The bins that are sought, by the whole work-group.
__device__ __forceinline__ Bins find_bins(const MyBins& my, const Setting& set, u64* mass_lds,
                                          uint32_t* count_lds, Bins& out) {
  constexpr int kEach = MyBins::kEach;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const u64* m = my.m;
  const uint32_t* n = my.n;
  u64 mass = 0;
  uint32_t count = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    mass += m[i];
    count += n[i];
  }
  u64 mass_to = wave_upto(mass);
  uint32_t count_to = wave_upto(count);
  if (lane == 63) {
    mass_lds[wave] = mass_to;
    count_lds[wave] = count_to;
  }
  if (tid == 0) out = Bins{-1, -1, -1, 0, 0, 0, 0};
  __syncthreads();
  u64 all = 0;
  mass_to -= mass;
  count_to -= count;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) {
      mass_to += mass_lds[w];
      count_to += count_lds[w];
    }
    all += mass_lds[w];
  }
  if (tid == 0) out.all = all;
  // the k-th token's bin; among tokens without a step there is nothing to cut
  if (set.cut_k) {
    uint32_t upto = count_to;
    u64 above = mass_to;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (upto < (uint32_t)set.k && (uint32_t)set.k <= upto + n[i]) {
        out.k = kEach * tid + i;
        out.above_k = upto;
        out.mass_above_k = above;
        mass_lds[kWaves] = above;
        mass_lds[kWaves + 1] = above + m[i];
      }
      upto += n[i];
      above += m[i];
    }
  }
  __syncthreads();
  if (set.cut_p) {
    // top_p of at least what lies above the k-th token's bin, and at most that and all of the bin
    const bool k_cuts = out.k >= 0;
    const u64 low = set.share_of(k_cuts ? mass_lds[kWaves] : all);
    const u64 high = set.share_of(k_cuts ? mass_lds[kWaves + 1] : all);
    u64 above = mass_to;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (above < low && low <= above + m[i]) {
        out.p_low = kEach * tid + i;
        out.mass_above_p = above;
      }
      if (above < high && high <= above + m[i]) out.p_high = kEach * tid + i;
      above += m[i];
    }
  }
  __syncthreads();
  return out;
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void sample_gather(SampleArgs p) {
  __shared__ u64 mass_lds[kWaves + 2], list[kList];
  __shared__ uint32_t count_lds[kWaves], listed, at_lds;
  __shared__ Bins bins_lds;
  const int slice = blockIdx.x, r = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Row<TYPE> row(p, r);
  constexpr int kLen = Row<TYPE>::kLen;
  int from, to;
  slice_of(p, row, slice, from, to);
  const u32x4 first = first_vector(row, from, to, wave, lane);
  const MyBins my(p, r, tid);
  const Setting set(p, r);
  const u64 best = row_best(p, r, lane);
  if (set.greedy || row_is_bad(best) || !(set.cut_k || set.cut_p)) return;
  if (tid == 0) listed = 0;
  const Bins bins = find_bins(my, set, mass_lds, count_lds, bins_lds);
  const float top = row_top(row, best);
  const uint32_t top_key = key_of(top);
  const Weights weights(top, set.t);
  const int first_bin = bins.first(), last_bin = max(bins.k, bins.p_high);
  // nothing below the last bin of the list is looked at
  const float least = last_bin >= 0 ? weights.logit_below((last_bin + 1) * (-1. / kBinsPerPower))
                                    : weights.least(set.min_p);
  if (slice == 0 && tid == 0) p.bins[r] = bins;
  each_chunk(row, from, to, wave, kWaves, lane, first, [&](int c, const float* z) {
    const int at = row.first(c, lane);
    double sum = 0.;
    u64 all = 0;
    const auto put = [&](int i) {
      const uint32_t n = atomicAdd(&listed, 1u);
      if (n < kList) list[n] = place_of(key_of(z[i]), at + i);
    };
    if (__ballot(largest<kLen>(z) >= least)) {
#pragma unroll
      for (int i = 0; i < kLen; ++i) {
        if (!(z[i] >= least)) continue;
        const double e = weights.exponent(z[i]);
        const int b = Weights::bin(e);
        if (b < first_bin) {
          if (!(set.min_p > 0.f) || min_keeps(e, key_of(z[i]), top_key, set.min_p))
            sum += Weights::steps_at(e);
        } else if (bins.lists(b)) {
          put(i);
        }
      }
      all = wave_sum(Weights::whole(sum));
    }
    if (lane == 0) p.chunk_mass[(int64_t)r * p.max_chunks + c] = all;
  });
  // the slice's list to the row's; one that is too long makes the row's too long
  __syncthreads();
  const uint32_t mine = listed;
  if (tid == 0 && mine)
    at_lds = atomicAdd(&p.listed[r], mine <= kList ? mine : (uint32_t)kList + 1);
  __syncthreads();
  if (mine <= kList)
    for (uint32_t i = tid; i < mine; i += kThreads)
      if (at_lds + i < kList) p.list[(int64_t)r * kList + at_lds + i] = list[i];
}

// The last token that stays, by its place.
struct Cut {
  uint32_t key;
  int index;
  __device__ bool keeps(uint32_t k, int at) const { return k > key || (k == key && at <= index); }
};

struct Shared {
  u64 mass[kMaxChunks];   // of chunks; and of keys' bytes while a cut is sought
  uint32_t count[kMaxChunks];
  u64 list[kList], list_mass[kList];  // places, and their steps of p
  u64 byte_mass[kPickThreads], wave_mass[kPickWaves + 1];
  uint32_t byte_count[kPickThreads];
  // found by one thread for all
  uint32_t key;
  int index;
  u64 above, total, place;
  uint32_t above_count;
};

// Exclusive prefix of x[0, n) in place by the first wave; the sum is returned to its lanes.
template <class T>
__device__ T wave_prefix(T* x, int n, int lane) {
  T sum = 0;
  for (int i = 0; i < n; i += 64) {
    const T mine = i + lane < n ? x[i + lane] : 0;
    const T upto = wave_upto(mine);
    if (i + lane < n) x[i + lane] = sum + upto - mine;
    sum += last_lane(upto);
  }
  return sum;
}

// The sum over the threads before this one; that over all of them in sums[kPickWaves].
__device__ __forceinline__ u64 block_prefix(u64 mine, u64* sums, int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  u64 upto = wave_upto(mine);
  __syncthreads();  // (the last call's sums are read)
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  u64 all = 0;
  upto -= mine;
#pragma unroll
  for (int w = 0; w < kPickWaves; ++w) {
    if (w < wave) upto += sums[w];
    all += sums[w];
  }
  if (tid == 0) sums[kPickWaves] = all;
  __syncthreads();
  return upto;
}

// A work-group a row.
template <int TYPE>
__global__ __launch_bounds__(kPickThreads) void sample_pick(SampleArgs p) {
  __shared__ Shared sh;
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int kThreads = kPickThreads, kWaves = kPickWaves;
  const Setting set(p, r);
  Row<TYPE> row(p, r);
  for (int c = tid; c < row.chunks; c += kThreads)
    sh.mass[c] = p.chunk_mass[(int64_t)r * p.max_chunks + c];
  const bool cuts = set.cut_k || set.cut_p;
  const uint32_t listed = p.listed[r];
  const float u = p.u[r];
  // (what no kernel has written for this row is not used)
  const Bins bins = p.bins[r];
  const u64 first_listed = p.list[(int64_t)r * kList + lane];
  const u64 best = row_best(p, r, lane);
  if (row_is_bad(best) || set.greedy) {
    if (tid == 0) {
      const bool bad = row_is_bad(best);
      p.ids[r] = bad ? -1 : token_at(best);
      if (p.logprob != nullptr) p.logprob[r] = bad ? __builtin_nanf("") : 0.f;
    }
    return;
  }
  constexpr int kLen = Row<TYPE>::kLen;
  float z[kLen];
  const float top = row_top(row, best);
  const uint32_t key = key_of(top);
  const Weights weights(top, set.t);

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
          atomicAdd(&sh.mass[255 - (k >> shift & 255)], weights.steps(z[i]));
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
    const u64 each = weights.steps(value_of(prefix));
    const u64 left = by_count ? target - above_count
                              : (each == 0 ? 1 : (target - above + each - 1) / each);
    __syncthreads();
    for (int c = wave; c < row.chunks; c += kWaves) {
      row.load(c, lane, z);
      const int first = row.first(c, lane);
      uint32_t n = 0;
#pragma unroll
      for (int i = 0; i < kLen; ++i) n += row.has(first + i) && key_of(z[i]) == prefix;
      n = wave_sum(n);
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
      uint32_t last = 0;
      for (int c = lane; c < row.chunks; c += 64)
        if (sh.count[c] < left) last = c;
      const int chunk = (int)wave_max(last);
      row.load(chunk, lane, z);
      const int first = row.first(chunk, lane);
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < kLen; ++i) mine += row.has(first + i) && key_of(z[i]) == prefix;
      const uint32_t upto = wave_upto(mine);
      u64 n = sh.count[chunk] + upto - mine;
#pragma unroll
      for (int i = 0; i < kLen; ++i)
        if (row.has(first + i) && key_of(z[i]) == prefix && ++n == left) sh.index = first + i;
    }
    __syncthreads();
    return Cut{prefix, sh.index};
  };

  Cut cut{0, row.vocab};
  const auto kept = [&](float v, int i) -> u64 {  // the steps of p where the token stays, else 0
    const uint32_t kk = key_of(v);
    const bool stays = row.has(i) && cut.keeps(kk, i) &&
                       (!(set.min_p > 0.f) || min_keeps(weights.exponent(v), kk, key, set.min_p));
    return stays ? weights.steps(v) : 0;
  };
  const auto chunk_sums = [&] {
    __syncthreads();
    for (int c = wave; c < row.chunks; c += kWaves) {
      row.load(c, lane, z);
      const int first = row.first(c, lane);
      u64 sum = 0;
#pragma unroll
      for (int i = 0; i < kLen; ++i) sum += kept(z[i], first + i);
      sum = wave_sum(sum);
      if (lane == 0) sh.mass[c] = sum;
    }
    __syncthreads();
  };

  if (cuts && listed > (uint32_t)kList) {
    u64 total = 0;
    if (set.cut_k) {
      cut = find_cut(true, (u64)set.k);
      total = sh.above;
    } else {
      total = bins.all;
    }
    if (set.cut_p) cut = find_cut(false, set.share_of(total));
    chunk_sums();
  } else {
    if (cuts && listed > 0) {
      const int n = (int)listed;
      const auto steps_of = [&](u64 place) {
        return weights.steps(value_of(key_at(place)));
      };
      const auto bin_of = [&](u64 place) {
        return Weights::bin(weights.exponent(value_of(key_at(place))));
      };
      const u64* places = p.list + (int64_t)r * kList;
      u64 place = 0;  // of the cut; 0: there is none
      if (n <= 64) {
        // every wave by itself: a lane an entry, which counts what is before it (seven rows with top_k:
        // 19.4 us, 22.4 by the bytes of the longer lists)
        const bool in = lane < n, in_k = in && bin_of(first_listed) == bins.k;
        const u64 x = in ? first_listed : 0, m = in ? steps_of(x) : 0;
        const u64 k_lanes = __ballot(in_k);
        u64 before = 0, before_k = 0;
        int rank_k = 0;
        for (int j = 0; j < n; ++j) {
          const u64 y = lane_at(x, j), mass = lane_at(m, j);
          const bool above = y > x, of_k = (k_lanes >> j) & 1;
          before += above ? mass : 0;
          before_k += above && of_k ? mass : 0;
          rank_k += above && of_k;
        }
        u64 total = bins.all;
        if (bins.k >= 0) {
          const u64 hit = __ballot(in_k && rank_k == set.k - (int)bins.above_k - 1);
          const int at = __builtin_ctzll(hit);
          place = lane_at(x, at);
          total = bins.mass_above_k + lane_at(before_k + m, at);
        }
        if (set.cut_p) {
          const u64 want = set.share_of(total), sum = bins.mass_above_p + before;
          const u64 hit = __ballot(in && sum < want && want <= sum + m);
          if (hit) place = lane_at(x, __builtin_ctzll(hit));
        }
        if (wave == 0 && in) sh.list[lane] = x;
      } else {
        u64 vary = 0;
        for (int i = tid; i < n; i += kThreads) {
          const u64 x = places[i];
          sh.list[i] = x;
          sh.list_mass[i] = steps_of(x);
          vary |= x ^ first_listed;
        }
        // (first_listed is another entry for each lane: the bits in which any two differ are among
        // these or in which those do)
        vary |= first_listed ^ lane_at(first_listed, 0);
        vary = wave_scan(vary, [](u64 a, u64 b) { return a | b; });
        if (lane == 63) sh.wave_mass[wave] = vary;
        __syncthreads();
        vary = 0;
        for (int w = 0; w < kWaves; ++w) vary |= sh.wave_mass[w];
        // The place at which the count or the sums of p of the entries, those of bin k alone or all,
        // pass a target; by the bytes in which entries differ, from the top, until one is left.  `sum`:
        // of p up to it.
        const auto find_place = [&](bool of_k, u64 target, u64& sum) -> u64 {
          u64 prefix = 0, above = 0;
          sum = 0;
          for (int shift = 56; shift >= 0; shift -= 8) {
            if (((vary >> shift) & 255) == 0) {
              prefix |= sh.list[0] & (255ull << shift);
              continue;
            }
            __syncthreads();
            sh.byte_mass[tid] = 0;
            sh.byte_count[tid] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kThreads) {
              const u64 x = sh.list[i];
              if (((x ^ prefix) & (~255ull << shift)) != 0 ||
                  (of_k && bin_of(x) != bins.k))
                continue;
              const int d = 255 - (int)(x >> shift & 255);
              atomicAdd(&sh.byte_count[d], 1u);
              atomicAdd(&sh.byte_mass[d], sh.list_mass[i]);
            }
            __syncthreads();
            const u64 mine = sh.byte_mass[tid], n_mine = sh.byte_count[tid];
            const u64 mass_before = block_prefix(mine, sh.wave_mass, tid);
            const u64 before = of_k ? block_prefix(n_mine, sh.wave_mass, tid) : mass_before;
            const u64 size = of_k ? n_mine : mine;
            if (above + before < target && target <= above + before + size) {
              sh.place = (u64)(255 - tid) << shift;
              sh.above = above + before;
              sh.total = sum + mass_before;
              sh.above_count = (uint32_t)n_mine;
            }
            __syncthreads();
            prefix |= sh.place;
            above = sh.above;
            sum = sh.total;
            if (sh.above_count == 1) {
              __syncthreads();  // (the byte is read)
              for (int i = tid; i < n; i += kThreads) {
                const u64 x = sh.list[i];
                if (((x ^ prefix) & (~0ull << shift)) == 0 && !(of_k && bin_of(x) != bins.k))
                  sh.place = x;
              }
              __syncthreads();
              return sh.place;
            }
          }
          return prefix;
        };
        u64 total = bins.all, sum;
        if (bins.k >= 0) {
          place = find_place(true, (u64)(set.k - (int)bins.above_k), sum);
          total = bins.mass_above_k + sum + steps_of(place);
        }
        if (set.cut_p) place = find_place(false, set.share_of(total) - bins.mass_above_p, sum);
      }
      if (place != 0) {
        cut = Cut{key_at(place), token_at(place)};
        __syncthreads();
        // what stays of the list joins its chunks
        for (int i = tid; i < n; i += kThreads) {
          const u64 x = sh.list[i];
          if (x < place) continue;
          const int at = token_at(x);
          atomicAdd(&sh.mass[(at + row.skew) / Row<TYPE>::kChunk],
                    kept(value_of(key_at(x)), at));
        }
      }
    }
    __syncthreads();
  }

  // the chunk in which the sum passes u of the whole
  const int each = (row.chunks + kThreads - 1) / kThreads, begin = tid * each;
  u64 mine = 0;
  for (int c = begin; c < min(begin + each, row.chunks); ++c) mine += sh.mass[c];
  u64 sum = block_prefix(mine, sh.wave_mass, tid);
  const u64 total = sh.wave_mass[kWaves];
  const double want = u > 0.f ? (double)u * (double)total : 0.;
  const u64 pass = want < (double)total ? min((u64)want, total - 1) : total - 1;
  if (sum <= pass && pass < sum + mine)
    for (int c = begin;; ++c) {
      if (pass < sum + sh.mass[c]) {
        sh.index = c;
        sh.above = sum;
        break;
      }
      sum += sh.mass[c];
    }
  __syncthreads();
  if (wave == 0) {
    const u32x4 w = row.raw(sh.index, lane);
    const double whole = log((double)total * 0x1p-44);  // (while the vector is in flight)
    row.take(w, z);
    const int first = row.first(sh.index, lane);
    u64 m[kLen], all = 0;
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      m[i] = kept(z[i], first + i);
      all += m[i];
    }
    const u64 upto = wave_upto(all);
    u64 at = sh.above + upto - all;
#pragma unroll
    for (int i = 0; i < kLen; ++i) {
      const u64 next = at + m[i];
      if (at <= pass && pass < next) {
        p.ids[r] = first + i;
        if (p.logprob != nullptr)
          p.logprob[r] = (float)(weights.exponent(z[i]) * 0.6931471805599453 - whole);
      }
      at = next;
    }
  }
}

}  // namespace

// Work-groups to a row: four of 512 threads on each CU in all, and a chunk at least for each wave (us
// with half, this and twice as many: 64 rows of 128000 51.5, 46.5, 53.3; 256 rows 112, 93.8, 90.6; 64
// of 8000 22 with any).
static int slices_of(int rows, int chunks) {
  return std::max(1, std::min({kMaxSlices, chunks / kWaves, 1024 / rows}));
}

static int chunks_of(int vocab, uint32_t flags) {
  const int chunk = (flags & WQ_FLAG_FP32) ? 256 : 512;
  return vocab / chunk + 2;  // (a row may begin and end inside one)
}

size_t sample_workspace_bytes(int rows, int vocab, uint32_t flags) {
  const size_t chunks = chunks_of(vocab, flags);
  return rows * (8 * (kMaxSlices + kBins + chunks + kList) + sizeof(Bins) + 4 * (kBins + 1));
}

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
  p.max_chunks = chunks_of(a.vocab, a.flags);
  p.slices = slices_of(a.rows, p.max_chunks);
  const size_t rows = a.rows;
  p.best = static_cast<u64*>(a.workspace);
  p.bin_mass = p.best + rows * kMaxSlices;
  p.chunk_mass = p.bin_mass + rows * kBins;
  p.list = p.chunk_mass + rows * p.max_chunks;
  p.bins = reinterpret_cast<Bins*>(p.list + rows * kList);
  p.bin_count = reinterpret_cast<uint32_t*>(p.bins + rows);
  p.listed = p.bin_count + rows * kBins;
  const dim3 grid((unsigned)p.slices, (unsigned)a.rows), block(kThreads);
  const dim3 pick((unsigned)a.rows), pick_block(kPickThreads);
  const bool cuts = a.top_k != nullptr || a.top_p != nullptr;
  const auto run = [&](auto type) {
    constexpr int TYPE = decltype(type)::value;
    hipLaunchKernelGGL((sample_max<TYPE>), grid, block, 0, stream, p);
    hipLaunchKernelGGL((sample_bins<TYPE>), grid, block, 0, stream, p);
    if (cuts) hipLaunchKernelGGL((sample_gather<TYPE>), grid, block, 0, stream, p);
    hipLaunchKernelGGL((sample_pick<TYPE>), pick, pick_block, 0, stream, p);
    return hipGetLastError();
  };
  if (a.flags & WQ_FLAG_FP32) return run(std::integral_constant<int, kFp32>());
  if (a.flags & WQ_FLAG_BF16) return run(std::integral_constant<int, kBf16>());
  return run(std::integral_constant<int, kFp16>());
}

}  // namespace wq
