// Attention of one new token per sequence over a paged cache of 4-bit codes (wq_paged_attention4).
//
// As in the 16-bit kernel, a work-group takes a range of the batch's positions for one KV head, its
// waves take tiles of positions in turn with a running maximum, sum and output of their own, and
// both products run on 16x16x32 MFMAs with the positions as rows, S^T = K Q^T and O^T = V^T P^T.
// What differs is that a row is codes c and, for each group g of the head, a scale and an offset:
//
//   k_j[i] = o_jg + s_jg c_ji:   q . k_j = sum_g s_jg (q . c_j)_g + o_jg (sum of q over g)
//   sum_j p_j v_j[i]            = sum_j (p_j s_jg) c_ji + sum_j p_j o_jg
//
// so codes go into the products as they are, and what belongs to a (position, group) is applied to
// the scores and to p, in fp32.  The sixteen columns of a product are query heads times groups:
// column (h, g) holds head h's query with all but g's elements zero, its scores' lanes add up over g,
// and its p is multiplied by g's scale alone.  A column then costs what it would without groups,
// and an output column holds all of the head's elements, of which those in g are used.
//
// K's codes become bytes (two instructions and a half for eight): 0 to 15 are, as E4M3 values, 2^-9 to
// 15 2^-9, which an MFMA of 8-bit operands takes with a block scale of 2^9.  Its other operand is q in
// three E4M3 pieces of four bits each, below a power of two of its column.  V's codes meet p, whose range no
// 8-bit type has: they become bf16 values of 16 + c, an instruction and a shift for two, and the offsets
// o - 16 s take the 16 off again; p s is cut into two bf16 parts, which keep 16 bits.
//
// V's codes need the positions along the register: the transposing read of 4-bit elements gives a
// lane 16 positions of one element, which serve two products.
//
// Long sequences of one set of columns are bound by memory (131072 positions of 8 KV heads of 128, groups
// of 64, slots before heads: 33.4 us in the kernel, 4.5 TB/s; with the join 40.8, and 38.1 heads before
// slots), two sets by instructions, some 760 vector ones and 88 MFMAs a tile (64 sequences of up to 8192,
// 64 heads, groups of 32: 103 us, 2.3 TB/s; fp16 104), short ones by latency (128 positions: 7.1 us).  Heads
// past 128, and one group in two sets, are short of registers: 40 of the 102 instances keep some in scratch
// memory, most where the head is no multiple of 32 (up to 105), those of 256 6 to 27.  16 sequences of up to
// 4096, 32 heads of 256 over 8: 57.8 us in groups of 32, 38.1 of 64 (fp16 60.7 and 42.4).
#pragma once

#include <type_traits>

#include "wq_attention.h"

namespace wq {

struct Attn4Args : AttnArgs {
  const uint32_t *k_pairs, *v_pairs;
  int64_t pair_page, pair_slot, pair_head;
  int group_size;
  int kv_group;       // query heads of a KV head (`group`: those of a work-group's NK)
  int short_strides;  // strides of pages and slots, and slots times strides, are below 2^32
};

constexpr int pow2_from(int x) { return x <= 1 ? 1 : x <= 2 ? 2 : x <= 4 ? 4 : 8; }

// How a KV head's query heads lie in columns.  Two KV heads share a set where both fit (`pairs`): a
// column then works on half of the rows, a position's rows of two heads, which may share lines, are
// read together, and positions are cut more finely (131072 positions of 8 KV heads of 128: 40.8 us,
// 43.7 by single heads, slots stored before heads; 38.1 either way, heads before slots.  Seven windows
// of 1000 over 12 heads of 80: 15.6 and 17.1).  Eight groups have no such instance.  Two sets where one
// does not hold the heads of one (they share the conversions, the reads and the addresses), as far as
// the registers go (64 sequences of up to 8192, 64 heads over 8, groups of 32: 102 us, 118 by single
// sets).
struct Columns {
  int kv_heads, sets;
  int heads_log2;  // query heads of a work-group, at most
};
inline Columns columns_of(int group, int kv_heads, int groups, int head_dim, bool pairs) {
  const int padded = pow2_from(groups);
  Columns c{1, 1, padded == 1 ? 4 : padded == 2 ? 3 : padded == 4 ? 2 : 1};
  if (pairs && kv_heads > 1 && groups < 8 && 2 * group * padded <= 16) {
    c.kv_heads = 2;
  } else if (head_dim <= 128 && group * padded > 16) {
    c.sets = 2;
    ++c.heads_log2;
  }
  return c;
}

// hipErrorNotSupported, and no launch, where there is no instance.
hipError_t launch_attn4_fp16(const Attn4Args& p, const Columns& c, dim3 grid, hipStream_t stream);
hipError_t launch_attn4_bf16(const Attn4Args& p, const Columns& c, dim3 grid, hipStream_t stream);

namespace {

// Positions of a wave's step: 64 rows of K and V, of one KV head or of two.
constexpr int tile_of(int nk) { return 64 / nk; }

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;

// Eight codes as 16 + c, nibbles in the order 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ bf16x8 from_codes(uint32_t w, uint32_t pattern) {
  const uint32_t mask = 0x00780078u;
  u32x4 x;
  x[0] = ((w << 3) & mask) | pattern;
  x[1] = ((w >> 1) & mask) | pattern;
  x[2] = ((w >> 5) & mask) | pattern;
  x[3] = ((w >> 9) & mask) | pattern;
  return __builtin_bit_cast(bf16x8, x);
}

__device__ __forceinline__ f32x4 mfma_bf(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float add_bits(float x, int y) {
  return x + __builtin_bit_cast(float, y);
}
// Sum over the groups' lanes of a head (GP neighbours).
template <int GP>
__device__ __forceinline__ float group_sum(float x) {
  if constexpr (GP >= 2)  // quad_perm 1 0 3 2
    x = add_bits(x, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0xB1, 0xf, 0xf, false));
  if constexpr (GP >= 4)  // quad_perm 2 3 0 1
    x = add_bits(x, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x4E, 0xf, 0xf, false));
  if constexpr (GP >= 8)  // row_half_mirror: the other four of eight lanes, whose sums are equal
    x = add_bits(x, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x141, 0xf, 0xf, false));
  return x;
}

// f over the four lanes of a column (16 apart): rows of 16 lanes change places in pairs.
template <class F>
__device__ __forceinline__ float over_column(float x, F f) {
  const auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x),
                                                  __builtin_bit_cast(uint32_t, x), false, false);
  x = f(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x),
                                                  __builtin_bit_cast(uint32_t, x), false, false);
  return f(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}
__device__ __forceinline__ float column_max(float x) {
  return over_column(x, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float column_sum(float x) {
  return over_column(x, [](float a, float b) { return a + b; });
}

// W: dwords of a row that a lane holds of K, head_dim rounded up over 32.  G: groups of a head.  NC:
// sets of sixteen columns that a work-group takes, which share K's and V's operands.  NK: KV heads that
// share a set: the first half of a tile's rows is one's, the second the other's, and a column looks at
// its own.  FULL: head_dim is 32 W.
template <bool BF16, int W, int G, int NC, int NK, bool FULL>
__global__ __launch_bounds__(kWaves * 64, 2) void attn4_kernel(Attn4Args p) {
  using A = Act<BF16>;
  static_assert(NK == 1 || NC == 1, "two KV heads take one set of columns");
  constexpr int DP = 32 * W;
  constexpr int GP = pow2_from(G);
  constexpr int kTile = tile_of(NK), kStep = kWaves * kTile;
  constexpr int NT = 4;                // 16-row blocks of a tile
  constexpr int NL = NT / NK;          // blocks that a column looks at
  constexpr int NB = DP / 16;          // 16-element blocks of the output
  constexpr int NM = (2 * W + 7) / 8;  // 128-element steps of K
  constexpr int NP = 3;                // pieces of q
  // Pieces in registers.  Where these are short the last ones lie in LDS and are read for each tile (us
  // with all in registers and so: 64 fp16 sequences of 64 heads of up to 8192, groups of 32, 125 and 104; 16
  // of up to 4096, heads of 256 in groups of 32 66.6 and 63.2, bf16 in one group 42.9 and 39.5; heads of 224
  // 87.7 and 71.5).  Not of one group in two sets (32 heads to a KV head, bf16: 38.6 and 43.2), nor of fp16
  // heads in one (of 200 46.8 and 50.1).
  constexpr int NR = NC == 2 && G > 1 ? 1 : W > 4 && (BF16 || G > 1) ? 2 : NP;
  constexpr int NA = NP - NR;
  constexpr int HS = 16 / GP;          // query heads of a set
  constexpr int HB = NC * HS;          // and of a work-group
  constexpr int SD = W % 2 == 0 ? 4 * W + 4 : 4 * W + 8;  // dwords of an LDS row of V: 4 mod 8
  constexpr int OS = DP + 4;           // LDS row of the joined outputs
  constexpr int kVDwords = 64 * SD + 2;
  constexpr int kVBytes = kWaves * kVDwords * 4, kOBytes = kWaves * HB * OS * 4;
  __shared__ __align__(16) uint8_t lds[kVBytes > kOBytes ? kVBytes : kOBytes];
  // scales and offsets of K, scales and offsets less 16 scales of V
  __shared__ __align__(16) float pair_lds[kWaves][4][G][64];
  __shared__ int64_t off_lds[kWaves][kTile];
  __shared__ float ml_lds[kWaves][HB][2];
  // q's last pieces: every wave writes the same, and a lane reads what it wrote.  Parts take turns,
  // because a wave that is done with one writes the next one's while others are still at it.
  __shared__ u32x4 last_lds[NA > 0 ? 2 : 1][NC][NM][NA > 0 ? NA : 1][2][64];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, qd = lane >> 4;
  int index, unit;
  if (!place_of_block(blockIdx.x, p.units, p.near_units != 0, p.ranges > 0 ? p.ranges : p.batch,
                      index, unit))
    return;
  Range rg{index, 0, 0};
  if (p.ranges > 0 && !find_range<kTile>(p, index, blockIdx.x == 0 && wave == 0, lane, rg)) return;
  const int kvh = unit / p.head_blocks, hb = unit - kvh * p.head_blocks;
  const int h0 = kvh * p.group + HB * hb;         // first query head
  const int rows = min(min(HB, p.group - HB * hb), p.q_heads - h0);
  const int my_head = row / GP, my_group = row % GP;  // this lane's column in a set
  const int my_kv = NK == 1 ? 0 : (int)(my_head >= p.kv_group);  // its KV head of the work-group's
  const int my_pair = GP == G ? my_group : min(my_group, G - 1);  // (no group: any pair will do)

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
    s.granules = granules_of<kTile>(p, len);
    s.count = p.ranges > 0 ? min(s.granules - first, left) : s.granules;
    const int start = window_start<kTile>(p, len);
    s.t0 = start + first * kStep;
    s.t1 = p.ranges > 0 ? min(len, start + (first + s.count) * kStep) : len;
    s.t_pages = p.ranges > 0 || p.window > 0 ? len : p.max_len;
    return s;
  };

  // A lane holds K's rows in pieces of four or two dwords, of which the four lanes of a row make a run.
  // Where the head ends inside one, a piece is read from as far before its place as it takes, and
  // what is there twice meets zeros of q the second time.
  constexpr int kPiece = W == 2 || W == 3 ? 2 : 4;
  constexpr auto kLength = [](int w) {  // of the piece that register w begins
    return W == 3 && w == 2 ? 1 : W == 6 && w == 4 ? 2 : kPiece;
  };
  const int nd = FULL ? 4 * W : p.d / 8;  // dwords of a row
  const auto place_of_piece = [&](int w) { return 4 * w + kLength(w) * qd; };
  const auto piece_at = [&](int w) {
    return FULL ? place_of_piece(w) : min(place_of_piece(w), nd - kLength(w));
  };

  // q as the B operand: this column's head, its group's elements, as pieces below 2^8 times the power
  // of two in q_scale; elements 0, 2, 4, 6 of a dword's eight, then the others, as K's bytes come.
  // The products of an 8-bit MFMA lose what lies more than ten bits below the largest operand's
  // exponent (measured: beside 128 a piece of 2^-4 counts for nothing), so a piece is a multiple of
  // 2^-3, whose products are whole, and what it leaves is the next one's, four bits down.  Three pieces
  // hold q to 2^-12 beside 2^7, two of bf16's to 2^-8, which showed in the log of the sum, by 1e-5.  (bf16
  // heads past 128 are faster with two, and what they leave met by the mean code: 16 sequences of up to
  // 4096, heads of 256 in groups of 32 56.9 us, 59.3 with three, of 64 39.3 and 38.6, in one group 35.3
  // and 39.6; heads of 192 28.6 and 29.6.)  A negative scale of the scores is q's sign, and one of 0 its
  // value.
  uint32_t pattern;
  asm volatile("v_mov_b32 %0, 0x41804180" : "=v"(pattern));
  const float sign = p.scale > 0.f ? 1.f : p.scale < 0.f ? -1.f : 0.f;
  const float sc = p.scale == 0.f ? 1.f : fabsf(p.scale);
  i32x8 qp[NC][NR][NM];
  int turn = 0;
  int q_scale[NC];
  float q_sum[NC];
  const auto element = [](u32x4 w, int t) { return A::value((uint16_t)(w[t / 2] >> (16 * (t % 2)))); };
  const auto load_q = [&](int b) {
    turn ^= 1;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int head = n * HS + my_head;
      const uint16_t* src = p.q + (int64_t)b * p.ldq + (int64_t)(h0 + (head < rows ? head : 0)) * p.d;
      u32x4 raw[W];
      float most = 0.f, sum = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const int first = w / kPiece * kPiece;
        const int dw = piece_at(first) + w - first;
        raw[w] = u32x4{0u, 0u, 0u, 0u};
        if ((FULL || dw >= place_of_piece(first)) && head < rows && 8 * dw / p.group_size == my_group)
          raw[w] = *reinterpret_cast<const u32x4*>(src + 8 * dw);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const float x = element(raw[w], t);
          sum += x;
          most = fmaxf(most, fabsf(x));
        }
      }
      q_sum[n] = sign * column_sum(sum);
      // the largest element's exponent, seven below which is the pieces' (within what scales hold);
      // one more where its first piece would round up to 2^8
      const float largest = column_max(most) * (256.f / 248.f);
      const int top = (int)(__builtin_bit_cast(uint32_t, largest) >> 23) - 127 - 7;
      const int e = min(max(top, -110), 120);
      q_scale[n] = 127 + e;
      const float down = __builtin_ldexpf(sign, -e);
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        i32x8 last[NA > 0 ? NA : 1];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int w = (8 * m + r) / 2, odd = r % 2;  // elements odd, odd + 2, ... of dword w
          float y[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) y[t] = w < W ? element(raw[w < W ? w : 0], 2 * t + odd) * down : 0.f;
#pragma unroll
          for (int piece = 0; piece < NP; ++piece) {
            float whole[4];  // of 2^-3
#pragma unroll
            for (int t = 0; t < 4; ++t) whole[t] = (y[t] + 0x1.8p20f) - 0x1.8p20f;
            int bytes = __builtin_amdgcn_cvt_pk_fp8_f32(whole[0], whole[1], 0, false);
            bytes = __builtin_amdgcn_cvt_pk_fp8_f32(whole[2], whole[3], bytes, true);
            if (piece < NR) {
              qp[n][piece < NR ? piece : 0][m][r] = bytes;
            } else {
              last[piece < NR ? 0 : piece - NR][r] = bytes;
            }
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(bytes, false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(bytes, true);
            y[0] = (y[0] - lo[0]) * 16.f;  // exact: what a piece leaves, four bits down
            y[1] = (y[1] - lo[1]) * 16.f;
            y[2] = (y[2] - hi[0]) * 16.f;
            y[3] = (y[3] - hi[1]) * 16.f;
          }
        }
#pragma unroll
        for (int k = 0; k < NA; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            last_lds[turn][n][m][k][i][lane] =
                u32x4{(uint32_t)last[k][4 * i], (uint32_t)last[k][4 * i + 1],
                      (uint32_t)last[k][4 * i + 2], (uint32_t)last[k][4 * i + 3]};
      }
    }
  };

  // the second KV head's rows; of an odd number of heads the last again, for columns without heads
  const int64_t second = NK == 2 && NK * kvh + 1 < p.kv_heads ? 1 : 0;
  const uint8_t* kbase = p.k + NK * kvh * p.head_stride / 2;
  const uint8_t* vbase = p.v + NK * kvh * p.head_stride / 2;
  const int64_t row_step = second * p.head_stride / 2;
  const int64_t pair_step = NK == 2 && lane >= 32 ? second * p.pair_head : 0;
  const uint32_t* k_pairs = p.k_pairs + NK * kvh * p.pair_head + pair_step;
  const uint32_t* v_pairs = p.v_pairs + NK * kvh * p.pair_head + pair_step;

  // Page numbers (and keep bytes) of the tile at t, one position per lane (NK 2: and half-wave).
  int page_next = -1, pos_next = 0, slot_next = 0;
  uint8_t keep_next = 1;
  const auto read_pages = [&](int b, int t_pages, int t) {
    const int pos = t + (lane & (kTile - 1));
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
  int64_t pair_off = 0;
  const auto place = [&](int lo, int t1) -> uint64_t {
    const bool live = (unsigned)page_next < (unsigned)p.num_pages && keep_next != 0 &&
                      pos_next >= lo && pos_next < t1;
    const int page = live ? page_next : 0, slot = live ? slot_next : 0;
    if (p.short_strides) {
      off_lds[wave][lane & (kTile - 1)] = (int64_t)(((uint64_t)(uint32_t)page * (uint32_t)p.page_stride +
                                       (uint32_t)slot * (uint32_t)p.slot_stride) /
                                      2);
      pair_off = (int64_t)((uint64_t)(uint32_t)page * (uint32_t)p.pair_page +
                           (uint32_t)slot * (uint32_t)p.pair_slot);
    } else {
      off_lds[wave][lane & (kTile - 1)] = (page * p.page_stride + slot * p.slot_stride) / 2;
      pair_off = page * p.pair_page + slot * p.pair_slot;
    }
    return __ballot(live);
  };
  uint32_t kr[NT][W], kp[G], vp[G];
  u32x4 vr[W];
  const auto load_k = [&] {
#pragma unroll
    for (int g = 0; g < G; ++g) kp[g] = k_pairs[pair_off + g];
#pragma unroll
    for (int blk = 0; blk < NT; ++blk) {
      const uint8_t* at = kbase + off_lds[wave][(16 * blk + row) & (kTile - 1)];
      if (NK == 2 && blk >= NL) at += row_step;
#pragma unroll
      for (int w = 0; w < W; w += kPiece) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(at) + piece_at(w);
#pragma unroll
        for (int i = 0; i < kLength(w); ++i) kr[blk][w + i] = src[i];
      }
    }
  };
  // V by whole rows, 16 bytes a lane: read once, so it need not stay in the caches.
  const auto load_v = [&] {
#pragma unroll
    for (int g = 0; g < G; ++g) vp[g] = v_pairs[pair_off + g];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const int piece = 64 * j + lane, r = piece / W, c = 4 * (piece % W);
      const uint32_t* at = reinterpret_cast<const uint32_t*>(
          vbase + off_lds[wave][r & (kTile - 1)] + (NK == 2 && r >= kTile ? row_step : 0));
      if (FULL || nd >= 4) {  // (the last piece of a row ends where the head does)
#pragma unroll
        for (int i = 0; i < 4; ++i) vr[j][i] = __builtin_nontemporal_load(at + min(c, nd - 4) + i);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) vr[j][i] = at[min(c + i, nd - 1)];
      }
    }
  };
  // Dword offset of V's row r in LDS: rows 4 qd + e of four blocks, 8 bytes each, that a transposing
  // read takes together, lie in different banks but for two blocks each.
  const auto v_row = [](int r) { return r * SD + 2 * (r >> 4 & 1); };
  // Pairs of the tile in LDS by group; zero where a position is not live, whatever lies there.
  const auto put_pairs = [&](uint64_t now) {
    const bool mine = (now >> lane) & 1;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t k = mine ? kp[g] : 0u, v = mine ? vp[g] : 0u;
      const float scale = A::value((uint16_t)v);
      pair_lds[wave][0][g][lane] = A::value((uint16_t)k);
      pair_lds[wave][1][g][lane] = A::value((uint16_t)(k >> 16));
      pair_lds[wave][2][g][lane] = scale;
      pair_lds[wave][3][g][lane] = __builtin_fmaf(-16.f, scale, A::value((uint16_t)(v >> 16)));
    }
  };
  const auto pairs_of = [&](int which, int blk) {  // (blk: of those that this column looks at)
    return *reinterpret_cast<const f32x4*>(
        &pair_lds[wave][which][my_pair][kTile * my_kv + 16 * blk + 4 * qd]);
  };

  uint32_t* const v_lds = reinterpret_cast<uint32_t*>(lds) + wave * kVDwords;
  const float sc2 = p.softcap > 0.f ? kLog2e : sc * kLog2e;  // scores to base 2
  const float cap = sc / p.softcap;
  uint64_t live = 0;
  bool ready = false;  // this part's first tile is requested, and the next one's pages are read
  bool first_part = true;
  Part cur = part_of(rg.b, rg.first, rg.left);

  for (;;) {
    rg.left -= cur.count;
    const bool more = p.ranges > 0 && rg.left > 0;
    Part nxt{};  // (no pages, nothing live)
    if (more) {
      int b = cur.b;
      do {  // (granules are left, so a sequence with some follows)
        ++b;
      } while (granules_of<kTile>(p, max(0, min(p.lens[b], p.max_len))) == 0);
      nxt = part_of(b, 0, rg.left);
    }
    const int b = cur.b;
    float m[NC], l[NC], low_sum[NC];  // m: of the scores before they are taken to base 2
    f32x4 o[NC][NB];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      m[n] = -INFINITY;
      l[n] = low_sum[n] = 0.f;
#pragma unroll
      for (int i = 0; i < NB; ++i) o[n][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // A wave's tiles follow each other from one part to the next, so that the next part's first is
    // in flight while the waves are joined.
    int t = cur.t0 + wave * kTile;
    const int next_t = nxt.t0 + wave * kTile, tiles = t >= cur.t1 ? 0 : t + kStep >= cur.t1 ? 1 : 2;
    if (!ready) {
      read_pages(cur.b, cur.t_pages, t);  // (without a tile: the cache's first slot)
      wave_lds_fence();
      live = place(cur.lo, cur.t1);
      wave_lds_fence();
      const bool here = tiles != 1;
      read_pages(here ? cur.b : nxt.b, here ? cur.t_pages : nxt.t_pages, here ? t + kStep : next_t);
      load_k();
      load_v();
    }
    if (first_part) load_q(cur.b);  // (behind the requests of the first tile)
    first_part = false;
    for (; t < cur.t1; t += kStep) {
      // the codes' products: what is not there of a row's last 128 elements meets zeros of q
      i32x8 last[NC][NM][NA > 0 ? NA : 1];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int j = 0; j < NM; ++j)
#pragma unroll
          for (int k = 0; k < NA; ++k)
#pragma unroll
            for (int r = 0; r < 8; ++r)
              last[n][j][k][r] = (int)last_lds[turn][n][j][k][r / 4][lane][r % 4];
      f32x4 all[NC][NT];
#pragma unroll
      for (int blk = 0; blk < NT; ++blk) {
#pragma unroll
        for (int n = 0; n < NC; ++n) all[n][blk] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NM; ++j) {
          i32x8 c;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const int w = (8 * j + r) / 2;
            c[r] = (int)(kr[blk][w < W ? w : 0] >> (r % 2 ? 4 : 0) & 0x0f0f0f0fu);
          }
#pragma unroll
          for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int piece = 0; piece < NP; ++piece)
              all[n][blk] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                  c, piece < NR ? qp[n][piece < NR ? piece : 0][j] : last[n][j][piece < NR ? 0 : piece - NR],
                  all[n][blk], 0, 0, 0, 127 + 9, 0, q_scale[n] - 4 * piece);
        }
      }
      f32x4 s[NC][NL];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int blk = 0; blk < NL; ++blk) {
          s[n][blk] = all[n][blk];
          if constexpr (NK == 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][blk][e] = my_kv ? all[n][blk + NL][e] : all[n][blk][e];
          }
        }
      const uint64_t now = live;
      put_pairs(now);
      // the next tile's K (positions past the range are not live and read the first slot)
      const bool ends = t + kStep >= cur.t1;
      wave_lds_fence();
      live = place(ends ? nxt.lo : cur.lo, ends ? nxt.t1 : cur.t1);
      wave_lds_fence();
      const bool here = t + 2 * kStep < cur.t1;
      read_pages(here ? cur.b : nxt.b, here ? cur.t_pages : nxt.t_pages,
                 here ? t + 2 * kStep : next_t + (ends ? kStep : 0));
      load_k();

      // scores: this column's group, then all of the head's
#pragma unroll
      for (int blk = 0; blk < NL; ++blk) {
        const f32x4 scale = pairs_of(0, blk), offset = pairs_of(1, blk);
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[n][blk][e] = group_sum<GP>(__builtin_fmaf(scale[e], s[n][blk][e], offset[e] * q_sum[n]));
      }
      if (p.softcap > 0.f) {
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int blk = 0; blk < NL; ++blk)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[n][blk][e] = capped(s[n][blk][e] * sc, s[n][blk][e] * cap, p.softcap);
      }
      if (now != ~0ull) {
        uint32_t lo = (uint32_t)now >> (4 * qd), hi = (uint32_t)(now >> 32) >> (4 * qd);
        if (NK == 2) hi = lo;  // (both KV heads' positions are the same)
#pragma unroll
        for (int blk = 0; blk < NL; ++blk)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // all ones where the position is live
            const uint32_t mine =
                (uint32_t)__builtin_amdgcn_sbfe((int)(blk < 2 ? lo : hi), 16 * (blk % 2) + e, 1);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
              const float x = s[n][blk][e];
              const uint32_t bits =
                  (__builtin_bit_cast(uint32_t, x) & mine) | (0xff800000u & ~mine);
              s[n][blk][e] = __builtin_bit_cast(float, bits);
            }
          }
      }

      // running maximum and sum
      float base[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        float mx = -INFINITY;
#pragma unroll
        for (int blk = 0; blk < NL; ++blk)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[n][blk][e]);
        const float m_new = fmaxf(m[n], column_max(mx));
        const float top = m_new == -INFINITY ? 0.f : m_new;  // nothing live so far
        if (__ballot(m_new > m[n])) {  // some head's maximum moved
          const float alpha = __builtin_amdgcn_exp2f((m[n] - top) * sc2);
          l[n] *= alpha;
          low_sum[n] *= alpha;
#pragma unroll
          for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][i][e] *= alpha;
        }
        m[n] = m_new;
        base[n] = -top * sc2;
      }

      // p times the scale of this column's group as two bf16 parts, cut off and rounded; element
      // 2 e + i of a product's eight is position e of block 2 k + i, as V's codes come
      bf16x8 ph[NC][2], pl[NC][2];
#pragma unroll
      for (int k = 0; k < NL / 2; ++k) {
        f32x4 scale[2], low[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          scale[i] = pairs_of(2, 2 * k + i);
          low[i] = pairs_of(3, 2 * k + i);
        }
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          u32x4 high;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float x =
                  __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][2 * k + i][e], sc2, base[n]));
              l[n] += x;
              low_sum[n] = __builtin_fmaf(x, low[i][e], low_sum[n]);
              y[i] = x * scale[i][e];
              const uint32_t bits = __builtin_bit_cast(uint32_t, y[i]) & 0xffff0000u;
              pl[n][k][2 * e + i] = (bf16)(y[i] - __builtin_bit_cast(float, bits));
            }
            high[e] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, y[1]),
                                            __builtin_bit_cast(uint32_t, y[0]), 0x07060302u);
          }
          ph[n][k] = __builtin_bit_cast(bf16x8, high);
        }
      }
      if constexpr (NK == 2) {  // a column's own KV head's rows alone
        const bf16x8 none = {};
        ph[0][1] = my_kv ? ph[0][0] : none;
        pl[0][1] = my_kv ? pl[0][0] : none;
        ph[0][0] = my_kv ? none : ph[0][0];
        pl[0][0] = my_kv ? none : pl[0][0];
      }

#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int piece = 64 * j + lane;
        uint32_t* at = v_lds + v_row(piece / W);
        if constexpr (FULL) {
          at += 4 * (piece % W);
          *reinterpret_cast<u32x2*>(at) = u32x2{vr[j][0], vr[j][1]};
          *reinterpret_cast<u32x2*>(at + 2) = u32x2{vr[j][2], vr[j][3]};
        } else {  // (where it was read; of a head of less than 32 elements the first piece holds all)
          at += nd >= 4 ? min(4 * (piece % W), nd - 4) : 4 * (piece % W);
#pragma unroll
          for (int i = 0; i < 4; ++i) at[i] = vr[j][i];
        }
      }
      wave_lds_fence();
      load_v();

      const uint32_t* src = v_lds + v_row(16 * (row >> 2) + 4 * qd + (row & 3));
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const i32x2 c =
            __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_i32x2*)(src + 2 * i));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bf16x8 v = from_codes((uint32_t)c[k], pattern);
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            o[n][i] = mfma_bf(v, ph[n][k], o[n][i]);
            o[n][i] = mfma_bf(v, pl[n][k], o[n][i]);
          }
        }
      }
      wave_lds_fence();
    }

    ready = more && tiles > (ready ? 1 : 0);
    if (more) load_q(nxt.b);

    // Join the waves, in wave order.
    __syncthreads();  // every wave is done with its V rows
    float* const o_lds = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const float sum = column_sum(l[n]), low = column_sum(low_sum[n]);
      const int head = n * HS + my_head;
      if (qd == 0 && my_group == 0) {
        ml_lds[wave][head][0] = m[n] * sc2;
        ml_lds[wave][head][1] = sum;
      }
#pragma unroll
      for (int i = 0; i < NB; ++i)
        if (16 * i / p.group_size == my_group)
          *reinterpret_cast<f32x4*>(o_lds + (wave * HB + head) * OS + 16 * i + 4 * qd) =
              f32x4{o[n][i][0] + low, o[n][i][1] + low, o[n][i][2] + low, o[n][i][3] + low};
    }
    __syncthreads();
    const int per_row = p.d / 4;
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
        const f32x4 x = *reinterpret_cast<const f32x4*>(o_lds + (w * HB + r) * OS + e);
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
        const float f = sum == 0.f ? 0.f : 1.f / sum;
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
    __syncthreads();  // the joined outputs are no longer read, nor this part's q
  }
}

template <bool BF16, int W, int G, bool FULL>
hipError_t launch_attn4_n(const Attn4Args& p, const Columns& c, dim3 grid, hipStream_t stream) {
  const dim3 block(kWaves * 64);
  if (c.kv_heads == 1 && c.sets == 1) {
    hipLaunchKernelGGL((attn4_kernel<BF16, W, G, 1, 1, FULL>), grid, block, 0, stream, p);
    return hipGetLastError();
  }
  if constexpr (G < 8) {
    if (c.kv_heads == 2 && c.sets == 1) {
      hipLaunchKernelGGL((attn4_kernel<BF16, W, G, 1, 2, FULL>), grid, block, 0, stream, p);
      return hipGetLastError();
    }
  }
  if constexpr (W <= 4) {
    if (c.kv_heads == 1 && c.sets == 2) {
      hipLaunchKernelGGL((attn4_kernel<BF16, W, G, 2, 1, FULL>), grid, block, 0, stream, p);
      return hipGetLastError();
    }
  }
  return hipErrorNotSupported;
}

// The instance for a head_dim: rounded up to 64, 96, 128, 192 and 256.  A head that is no multiple of 32
// is one group, but for 160 and 224.
template <bool BF16, int W>
hipError_t launch_attn4_w(const Attn4Args& p, const Columns& c, dim3 grid, hipStream_t stream) {
  const int groups = p.d / p.group_size;
  if (p.d != 32 * W) {
    if (groups == 1) return launch_attn4_n<BF16, W, 1, false>(p, c, grid, stream);
    if constexpr (W == 6) {
      if (groups == 5) return launch_attn4_n<BF16, W, 5, false>(p, c, grid, stream);
    }
    if constexpr (W == 8) {
      if (groups == 7) return launch_attn4_n<BF16, W, 7, false>(p, c, grid, stream);
    }
    return hipErrorNotSupported;
  }
  if (groups == 1) return launch_attn4_n<BF16, W, 1, true>(p, c, grid, stream);
  if constexpr (W == 2 || W == 4 || W == 8) {
    if (groups == 2) return launch_attn4_n<BF16, W, 2, true>(p, c, grid, stream);
  }
  if constexpr (W == 4 || W == 8) {
    if (groups == 4) return launch_attn4_n<BF16, W, 4, true>(p, c, grid, stream);
  }
  if constexpr (W == 8) {
    if (groups == 8) return launch_attn4_n<BF16, W, 8, true>(p, c, grid, stream);
  }
  if constexpr (W == 3 || W == 6) {
    if (groups == 3) return launch_attn4_n<BF16, W, 3, true>(p, c, grid, stream);
  }
  if constexpr (W == 6) {
    if (groups == 6) return launch_attn4_n<BF16, W, 6, true>(p, c, grid, stream);
  }
  return hipErrorNotSupported;
}

template <bool BF16>
hipError_t launch_attn4(const Attn4Args& p, const Columns& c, dim3 grid, hipStream_t stream) {
  if (p.d <= 64) return launch_attn4_w<BF16, 2>(p, c, grid, stream);
  if (p.d <= 96) return launch_attn4_w<BF16, 3>(p, c, grid, stream);
  if (p.d <= 128) return launch_attn4_w<BF16, 4>(p, c, grid, stream);
  if (p.d <= 192) return launch_attn4_w<BF16, 6>(p, c, grid, stream);
  return launch_attn4_w<BF16, 8>(p, c, grid, stream);
}

}  // namespace
}  // namespace wq
