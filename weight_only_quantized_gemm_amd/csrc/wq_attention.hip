// Attention of one new token per sequence over a paged KV cache (wq_paged_attention).
//
// Each live K and V element is read once and takes part in 2 * (query heads per KV head)
// products, so the kernel is bound by the cache reads.  The batch's positions are cut into ranges
// of one length (a range a sequence where these are short); a work-group takes a range for one KV
// head and up to 16 of its query heads.  Its waves take tiles of 32 or 64 positions in turn and
// keep their own running maximum, sum and output, joined at the end of each sequence through LDS.
// Sequences that lie in several ranges leave fp32 partials that attn_join_kernel adds in their
// order.
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
// are formed, V when this tile's V has gone to LDS, and page numbers are read a tile further
// ahead.  As compiled, a tile's first score waits for its V and the next pages as well as for its
// K (on one path into the loop Q is the newest load), so nothing is in flight while scores are
// formed.
//
// Measured as a graph, and in a kernel trace, 8 KV heads of 128: one sequence of 131072 positions,
// bf16, 92 us, 5.8 TB/s, or 97, by where in memory the cache lies (89.8 us and the join's 4.8; the
// matrix units are busy 6% of the time); 16 sequences of up to 4096, 30 us, 4.8 TB/s (27.6, and
// 4.3); 64 of up to 8192, E4M3, 70% of the positions kept, 85 us, 4.4 TB/s of the kept rows (79.0,
// and 5.9; matrix units 15%, dropped rows and conversions between); one sequence of 128: 5.8 us,
// the launch and two trips to memory, for the page and for K and V.  No byte is fetched twice: the
// counters show 153.1 MB for the 152.6 of the live rows of 16 sequences, 375.0 for 370.7 kept
// ones of 64, and 21.1 for the 20.8 inside the windows of seven of up to 3001.
#include <algorithm>
#include <type_traits>

#include "wq_attention.h"

namespace wq {
namespace {

constexpr int kBlockShift = 4;  // 16 query heads to a work-group

// Positions of a wave's step (dp: head_dim rounded up to 64, 128 or more).  64 rows of an E4M3
// head of 128 keep 16 KiB requested, as 32 of a 16-bit one do (16 sequences of 4096 positions:
// 36.4 us with 32, 34.7 with 64; one of 65536: 35.3 and 32.7).  16-bit heads of 64 are faster
// with 32, whose registers leave room for a third work-group on the CU.
constexpr int tile_of(int dp, bool kv8) { return kv8 && dp <= 128 ? 64 : 32; }
// Binary places p is raised by (its maximum is 2^kPShift).
template <bool BF16>
constexpr float kPShift = BF16 ? 0.f : 15.f;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <bool BF16>
__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return Act<BF16>::mfma16(a, __builtin_bit_cast(typename Act<BF16>::W8, b), c);
}

template <bool BF16>
__device__ __forceinline__ f16x8 from_e4m3(uint32_t lo, uint32_t hi) {
  return __builtin_bit_cast(f16x8, Act<BF16>::fp8(lo, hi));
}

// Eight values >= 0 as high + low 16-bit parts.
template <bool BF16>
__device__ __forceinline__ void split_p(const float* p, f16x8& high, f16x8& low) {
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = p[2 * i], y = p[2 * i + 1];
    if constexpr (BF16) {
      const uint32_t xb = __builtin_bit_cast(uint32_t, x) & 0xffff0000u;
      const uint32_t yb = __builtin_bit_cast(uint32_t, y) & 0xffff0000u;
      hi[i] = xb >> 16 | yb;
      const float xl = fmaxf(x - __builtin_bit_cast(float, xb), 0x1p-100f);
      const float yl = fmaxf(y - __builtin_bit_cast(float, yb), 0x1p-100f);
      lo[i] = (uint32_t)Act<true>::round(xl) | (uint32_t)Act<true>::round(yl) << 16;
    } else {
      const auto h = __builtin_amdgcn_cvt_pkrtz(x, y);
      hi[i] = __builtin_bit_cast(uint32_t, h);
      const auto r = __builtin_amdgcn_cvt_pkrtz(fmaxf(x - (float)h[0], 0x1p-24f),
                                                fmaxf(y - (float)h[1], 0x1p-24f));
      lo[i] = __builtin_bit_cast(uint32_t, r);
    }
  }
  __builtin_memcpy(&high, hi, 16);
  __builtin_memcpy(&low, lo, 16);
}

// DP: head_dim rounded up (launch_attn); FULL: head_dim is DP.
template <bool BF16, bool KV8, int DP, bool FULL>
__global__ __launch_bounds__(kWaves * 64) void attn_kernel(AttnArgs p) {
  using A = Act<BF16>;
  constexpr int TILE = tile_of(DP, KV8), kStep = kWaves * TILE;
  constexpr int NT = TILE / 16;          // 16-position blocks of a tile
  constexpr int NS = DP / 32;            // MFMA steps along the head
  constexpr int NK = KV8 ? NS / 2 : NS;  // 16-byte K vectors per lane and position block
  constexpr int CE = KV8 ? 16 : 8;       // elements of a 16-byte vector
  constexpr int CPR = DP / CE;           // vectors of a V row
  constexpr int NV = TILE * CPR / 64;    // V vectors per lane
  constexpr int NB = DP / 16;            // 16-element blocks of the output
  constexpr int VS = DP + 16;            // LDS row of V: rows start 8 banks apart, or more
  constexpr int OS = DP + 4;             // LDS row of the joined outputs
  constexpr int kVBytes = kWaves * TILE * VS * 2, kOBytes = kWaves * 16 * OS * 4;
  __shared__ __align__(16) uint8_t lds[kVBytes > kOBytes ? kVBytes : kOBytes];
  __shared__ int64_t off_lds[kWaves][TILE];
  __shared__ float ml_lds[kWaves][16][2];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, qd = lane >> 4;
  int index, unit;
  if (!place_of_block(blockIdx.x, p.units, p.near_units != 0, p.ranges > 0 ? p.ranges : p.batch,
                      index, unit))
    return;
  Range rg{index, 0, 0};
  if (p.ranges > 0 && !find_range<TILE>(p, index, blockIdx.x == 0 && wave == 0, lane, rg)) return;
  const int kvh = unit / p.head_blocks, hb = unit - kvh * p.head_blocks;
  const int h0 = kvh * p.group + 16 * hb;         // first query head
  const int rows = min(16, p.group - 16 * hb);

  // Part of a sequence that this range holds.
  struct Part {
    int b, lo, t0, t1;           // sequence, first live position, positions [t0, t1)
    int t_pages;                 // page numbers are read for positions below it
    int first, count, granules;  // granules of the sequence: first one here, how many, in all
  };
  const auto part_of = [&](int b, int first, int left) {
    Part s;
    const int len = max(0, min(p.lens[b], p.max_len));
    s.b = b;
    s.lo = p.window > 0 ? max(0, len - p.window) : 0;
    s.first = first;
    s.granules = granules_of<TILE>(p, len);
    s.count = p.ranges > 0 ? min(s.granules - first, left) : s.granules;
    const int start = window_start<TILE>(p, len);
    s.t0 = start + first * kStep;
    s.t1 = p.ranges > 0 ? min(len, start + (first + s.count) * kStep) : len;
    // without ranges or a window they need not wait for the length
    s.t_pages = p.ranges > 0 || p.window > 0 ? len : p.max_len;
    return s;
  };

  // Q as the B operand; query heads past the last repeat the first (never stored).
  f16x8 qf[NS];
  const auto load_q = [&](int b) {
    const uint16_t* qp = p.q + (int64_t)b * p.ldq + (int64_t)(h0 + (row < rows ? row : 0)) * p.d;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int e = KV8 ? 64 * (s / 2) + 16 * qd + 8 * (s % 2) : 32 * s + 8 * qd;
      qf[s] = f16x8{};
      if (FULL || e < p.d) qf[s] = *reinterpret_cast<const f16x8*>(qp + e);
    }
  };

  const uint8_t* kbase = p.k + kvh * p.head_stride * (KV8 ? 1 : 2);
  const uint8_t* vbase = p.v + kvh * p.head_stride * (KV8 ? 1 : 2);

  // A vector that lies past the head's end is read from its start and not used; an E4M3
  // vector that passes the end half way (head_dim % 16 == 8) is read 8 bytes earlier and
  // shifted.
  const auto vec_at = [&](int e) {
    return FULL || e + CE <= p.d ? e : (e < p.d ? p.d - CE : 0);
  };
  const auto vec_fix = [&](u32x4 w, int e) {
    if (FULL) return w;
    if (KV8 && e < p.d && e + CE > p.d) w = u32x4{w[2], w[3], 0u, 0u};
    return e < p.d ? w : u32x4{0u, 0u, 0u, 0u};
  };

  // Page numbers (and keep bytes) of the tile at t, one position per lane and half-wave.
  int page_next = -1, pos_next = 0, slot_next = 0;
  uint8_t keep_next = 1;
  const auto read_pages = [&](int b, int t_pages, int t) {
    const int pos = t + (lane & (TILE - 1));
    const int at = (int)(__umulhi(2u * (unsigned)pos, p.page_mul) >> p.page_shift);
    pos_next = pos;
    slot_next = pos - at * p.page_size;
    page_next = -1;
    if (pos < t_pages) {
      page_next = p.table[(int64_t)b * p.table_stride + at];
      if (p.keep != nullptr) keep_next = p.keep[(int64_t)b * p.keep_stride + pos];
    }
  };
  // Cache offsets of the tile whose pages were read; returns the mask of live positions.  A
  // position that is not live reads the cache's first slot, and is not used.
  const auto place = [&](int lo, int t1) -> uint64_t {
    const bool live = (unsigned)page_next < (unsigned)p.num_pages && keep_next != 0 &&
                      pos_next >= lo && pos_next < t1;
    off_lds[wave][lane & (TILE - 1)] =
        live ? page_next * p.page_stride + slot_next * p.slot_stride : 0;
    return __ballot(live);
  };
  u32x4 kr[NT][NK], vr[NV];
  const auto load_k = [&] {
#pragma unroll
    for (int blk = 0; blk < NT; ++blk) {
      const uint8_t* kp = kbase + off_lds[wave][16 * blk + row] * (KV8 ? 1 : 2);
#pragma unroll
      for (int s = 0; s < NK; ++s)
        kr[blk][s] = *reinterpret_cast<const u32x4*>(
            kp + vec_at(4 * CE * s + CE * qd) * (KV8 ? 1 : 2));
    }
  };
  // V is read once and by whole rows, so it need not stay in the caches (16 sequences of up to
  // 4096: 34.1 us, 30.0 so; 64 of 8192, 373 and 337).  A 64-byte piece of K's rows is followed by
  // the rest of its line, which has to be there still (one sequence of 131072 slot-major
  // positions: 99.0 us, V read so 91.0, both 100.8).
  const auto load_v = [&] {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      vr[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(
          vbase + (off_lds[wave][(64 * j + lane) / CPR] + vec_at(CE * ((64 * j + lane) % CPR))) *
                      (KV8 ? 1 : 2)));
  };

  uint16_t* const v_lds = reinterpret_cast<uint16_t*>(lds) + wave * TILE * VS;
  const float kscale = KV8 && p.k_scale != nullptr ? p.k_scale[kvh] : 1.f;
  const float sc = p.scale * kscale;
  const float sc2 = p.softcap > 0.f ? kLog2e : sc * kLog2e;
  const float cap = sc / p.softcap;
  uint64_t live = 0;
  bool ready = false;  // this part's first tile is requested, and the next one's pages are read
  Part cur = part_of(rg.b, rg.first, rg.left);
  load_q(cur.b);

  for (;;) {
    rg.left -= cur.count;
    const bool more = p.ranges > 0 && rg.left > 0;
    Part nxt{};  // (no pages, nothing live)
    if (more) {
      int b = cur.b;
      do {  // (granules are left, so a sequence with some follows)
        ++b;
      } while (granules_of<TILE>(p, max(0, min(p.lens[b], p.max_len))) == 0);
      nxt = part_of(b, 0, rg.left);
    }
    const int b = cur.b;
    float m = -INFINITY, l = 0.f;
    f32x4 o[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};

    // A wave's tiles follow each other from one part to the next: a part's last tiles request the
    // next one's first, so that it is in flight while the waves are joined (64 sequences of up to
    // 8192, E4M3, masked: 87.2 us without, 85.0 so; 100 of up to 1500 65.9, 63.4; a single part
    // pays 1% for the choices).  Only a wave with less than two tiles here may have none
    // requested.
    int t = cur.t0 + wave * TILE;
    const int next_t = nxt.t0 + wave * TILE, tiles = t >= cur.t1 ? 0 : t + kStep >= cur.t1 ? 1 : 2;
    if (!ready) {
      read_pages(cur.b, cur.t_pages, t);  // (without a tile: the cache's first slot)
      wave_lds_fence();
      live = place(cur.lo, cur.t1);
      wave_lds_fence();
      const bool here = tiles != 1;
      read_pages(here ? cur.b : nxt.b, here ? cur.t_pages : nxt.t_pages,
                 here ? t + kStep : next_t);
      load_k();
      load_v();
    }
    for (; t < cur.t1; t += kStep) {
      // scores
      f32x4 s[NT];
#pragma unroll
      for (int blk = 0; blk < NT; ++blk) {
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
      const uint64_t now = live;
      // the next tile's K (positions past the range are not live and read the first slot)
      const bool last = t + kStep >= cur.t1;
      wave_lds_fence();
      live = place(last ? nxt.lo : cur.lo, last ? nxt.t1 : cur.t1);
      wave_lds_fence();
      const bool here = t + 2 * kStep < cur.t1;
      read_pages(here ? cur.b : nxt.b, here ? cur.t_pages : nxt.t_pages,
                 here ? t + 2 * kStep : next_t + (last ? kStep : 0));
      load_k();

      // running maximum and sum, in base 2
      float mx = -INFINITY;
      if (p.softcap > 0.f) {
#pragma unroll
        for (int blk = 0; blk < NT; ++blk)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[blk][e] = capped(s[blk][e] * sc, s[blk][e] * cap, p.softcap);
      }
#pragma unroll
      for (int blk = 0; blk < NT; ++blk)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[blk][e] *= sc2;
      if (now != ~0ull) {
#pragma unroll
        for (int blk = 0; blk < NT; ++blk)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[blk][e] = (now >> (16 * blk + 4 * qd + e)) & 1 ? s[blk][e] : -INFINITY;
      }
#pragma unroll
      for (int blk = 0; blk < NT; ++blk)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[blk][e]);
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float m_new = fmaxf(m, mx);
      const float top = m_new == -INFINITY ? 0.f : m_new;  // nothing live so far
      const float ref = top - kPShift<BF16>;
      const float alpha = __builtin_amdgcn_exp2f(m - top);
      if (__ballot(m_new > m)) {  // some head's maximum moved
        l *= alpha;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= alpha;
      }
      m = m_new;
      // high + low: the high part is cut off, not rounded, so that the low part is never
      // negative, and it is kept above 0 (by 2^-39 of the largest p at most): an infinite value
      // of V then stays infinite
      f16x8 ph[NT / 2], pl[NT / 2];
#pragma unroll
      for (int k = 0; k < NT / 2; ++k) {
        float ps[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ps[i] = __builtin_amdgcn_exp2f(s[2 * k + i / 4][i % 4] - ref);
          l += ps[i];
        }
        split_p<BF16>(ps, ph[k], pl[k]);
      }

      // V to LDS as 16-bit rows, zero where a position is not live
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int r = (64 * j + lane) / CPR, vcol = CE * ((64 * j + lane) % CPR);
        u32x4 w = vec_fix(vr[j], vcol);
        if (now != ~0ull && !((now >> r) & 1)) w = u32x4{0u, 0u, 0u, 0u};
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
#pragma unroll
        for (int k = 0; k < NT / 2; ++k) {
          const s16x4 a0 =
              __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(src + 32 * k * VS));
          const s16x4 a1 =
              __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(src + (32 * k + 16) * VS));
          f16x8 vf;
          __builtin_memcpy(&vf, &a0, 8);
          __builtin_memcpy(reinterpret_cast<char*>(&vf) + 8, &a1, 8);
          o[i] = mfma<BF16>(vf, ph[k], o[i]);
          o[i] = mfma<BF16>(vf, pl[k], o[i]);
        }
      }
      wave_lds_fence();
    }

    ready = more && tiles > (ready ? 1 : 0);
    if (more) load_q(nxt.b);

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
      if (cur.count < cur.granules) {
        // a sequence that began in an earlier range leaves the range's first partial, one that
        // goes on in the next its second
        const int64_t part = 2 * index + (cur.first == 0);
        const int64_t at = (part * p.units + unit) * p.part_rows + r;
        *reinterpret_cast<f32x4*>(p.part_o + at * p.d + e) = acc;
        if (e == 0) {
          p.part_ml[at * 2] = top;
          p.part_ml[at * 2 + 1] = sum;
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
    if (!more) return;
    cur = nxt;
    __syncthreads();  // the joined outputs are no longer read
  }
}

// The instance for a head_dim.  Rounded up to 64 and to powers of two from there; 96 and 192 as
// well, where the rest of the next power of two costs registers, LDS and loads (16 sequences of up
// to 4096, us with 128 or 256 and so: heads of 80 26.0, 25.0; 96 27.5, 25.2; 192 52.3, 46.2, E4M3
// 32.5, 28.6; 160 46.7, 47.4).  A step of the head is 64 elements of an E4M3 row: no 96 there.
template <bool BF16, bool KV8>
void launch_attn(const AttnArgs& p, dim3 grid, hipStream_t stream) {
  const auto run = [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    const dim3 block(kWaves * 64);
    if (p.d == DP)
      hipLaunchKernelGGL((attn_kernel<BF16, KV8, DP, true>), grid, block, 0, stream, p);
    else
      hipLaunchKernelGGL((attn_kernel<BF16, KV8, DP, false>), grid, block, 0, stream, p);
  };
  if (p.d <= 64) return run(std::integral_constant<int, 64>());
  if constexpr (!KV8) {
    if (p.d <= 96) return run(std::integral_constant<int, 96>());
  }
  if (p.d <= 128) return run(std::integral_constant<int, 128>());
  if (p.d <= 192) return run(std::integral_constant<int, 192>());
  run(std::integral_constant<int, 256>());
}

}  // namespace

// Work-groups to cut the batch for.  A single sequence is cut evenly, into as many as hold the
// bytes in flight that the memory needs, 64 KiB on each CU (bf16, head_dim 128, 131072
// positions: 256 work-groups 91.0 us, 512 95.2, 1024 97.9; head_dim 64 54.6, 49.7, 55.9).  Several
// sequences' ranges begin and end inside sequences, so there are as many as the CUs hold at once
// by their registers (16 sequences of up to 4096: 256 work-groups 32.4 us, 512 30.1, 768 35.6;
// E4M3, 64 of up to 8192, masked: 256 109.1, 512 87.4, 768 103.2; head_dim 256: 57.9, 61.1, 70.3,
// E4M3 62.2, 58.5, 65.5; head_dim 64: 65.8, 54.8, 54.7).
int attn_groups(int batch, int head_dim, bool kv8) {
  if (batch == 1) return head_dim <= 64 ? 512 : 256;
  return head_dim <= 64 ? 768 : head_dim <= 128 || kv8 ? 512 : 256;
}

AttnPlan attn_plan(int batch, int q_heads, int kv_heads, int head_dim, int max_len, int window,
                   bool kv8) {
  AttnPlan plan{};
  plan.block_shift = kBlockShift;
  plan.head_blocks = (q_heads / kv_heads + 15) / 16;
  plan.units = kv_heads * plan.head_blocks;
  // positions a sequence may need, from the tile that holds the window's first
  const int tile = tile_of(head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256, kv8);
  const long span = window > 0 && window < max_len - tile ? window + tile - 1 : max_len;
  // Short sequences stay whole, which spares the partials and the join.  A work-group takes
  // about 1.2 us for 32 KiB of keys, so the longest there may be is bounded: a KiB of keys for
  // each work-group of the launch, between 96 and 256 (head_dim 128, 16-bit: 8 work-groups, 384
  // positions 9.4 us cut, 7.9 whole, 768 positions 9.4 and 11.5; 192 and 768: 20.9, 15.4; 512
  // and 1024: 52.0, 49.5; 8192 and 150: 194, 150).
  const long keys = span * head_dim * (kv8 ? 1 : 2);
  const long whole = std::min(256l, std::max(96l, (long)batch * plan.units)) * 1024;
  if (span > kWaves * tile && keys > whole) {
    const int groups = attn_groups(batch, head_dim, kv8);
    plan.ranges = groups / plan.units > 0 ? groups / plan.units : 1;
  }
  return plan;
}

size_t attn_workspace_bytes(const AttnPlan& plan, int batch, int q_heads, int kv_heads,
                            int head_dim) {
  if (plan.ranges == 0) return 0;
  const int group = q_heads / kv_heads;
  const size_t rows =
      2 * (size_t)plan.ranges * plan.units * std::min(group, 1 << plan.block_shift);
  return rows * (head_dim + 2) * sizeof(float) + 2 * (size_t)batch * sizeof(int32_t);
}

hipError_t launch_paged_attention(const wq_attn_args& a, const AttnPlan& plan,
                                  hipStream_t stream) {
  AttnArgs p = attn_args(a, plan, a.q_heads / a.cache.kv_heads);
  const bool bf16 = (a.flags & WQ_FLAG_BF16) != 0, kv8 = (a.flags & WQ_FLAG_FP8) != 0;
  // Work-groups go to the eight XCDs in turn.  Where several blocks of query heads read the same
  // rows, or the heads of a slot lie side by side in rows that do not end with a line, the units of
  // a range follow each other by eight, and the second finds the line in its L2 (16 sequences of
  // up to 4096, us before and with this: 32 query heads to a KV head 54.4, 45.7; slot-major heads
  // of 80 32.3, 28.6, E4M3 31.6, 27.1; one sequence of 100000, 128 query heads 66.6, 47.8).  Other
  // units share nothing, and are faster spread out (a slot-major sequence of 131072: 99.0, 102.7).
  p.near_units = plan.head_blocks > 1 || (p.kv_heads > 1 && p.head_stride < p.slot_stride &&
                                          p.head_stride * (kv8 ? 1 : 2) % 128 != 0);
  const dim3 grid = attn_grid(p);
  if (bf16)
    kv8 ? launch_attn<true, true>(p, grid, stream) : launch_attn<true, false>(p, grid, stream);
  else
    kv8 ? launch_attn<false, true>(p, grid, stream) : launch_attn<false, false>(p, grid, stream);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.ranges == 0) return e;
  return launch_attn_join<kBlockShift>(p, bf16, stream);
}

}  // namespace wq
