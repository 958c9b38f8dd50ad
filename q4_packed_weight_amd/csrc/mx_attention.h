// mx_attention.h -- what the attention kernels share: a sequence's rows and
// the keys they see, the fp16 operands made of queries and of cached blocks,
// and the joining of partial results.
//
// Operands.  Everything is multiplied in fp16 with powers of two taken out:
//   queries  q = 2^e (h + l): e by row, so that the row's largest value lies in
//            [2^14, 2^15); h alone holds bf16 and fp16 values, of fp32 h is
//            rounded to fp16 and l what is left, rounded too (off by 2^-23 of
//            the value).  Both end at fp16's smallest step, 2^-24: off by 2^-39 of
//            the row's largest, which bf16 and fp16 values notice from 2^-28 of it
//            down, and the l of fp32 from 2^-16.
//   keys and values  code * 2^(s - ref), ref the largest scale byte among the
//            keys taken together or up to 8 above it, so that the largest code
//            still fits: exact for blocks whose scale lies up to 2^21 (MX_FP8) or
//            2^36 (MX_FP4) below ref, as fp16's subnormals reach, and these
//            operands keep them.
//   weights  p = exp2(x - m), m 10 below the largest x so far or up to 4 less, so p at
//            most 2^14: one fp16, off by 2^-11 of p, an eighth of what bf16 would
//            leave of it; for fp32 a second one for what is left (2^-23); as fp16's
//            steps end, either by 2^-25 as well, 2^-35 of the largest, and below that
//            p is 0.  The sums of p are of the unrounded ones, in fp32.
// Keys that some rows see and others do not (a causal chunk's own, a window's
// edge) are taken without a common reference, which a key that a row does not
// see would give it: each key's own for its scores, and bf16 for its values (times
// 2^-8, so that the largest block is finite: nothing else keeps it from rows that do
// not see it), with one bf16 weight more, which takes the sums' power.
// The powers of q, k and scale are added as numbers before one of them is applied,
// so that a score is what its product says also where its factors are not near 1.
// A NaN block's scale is NaN and so are its products; a row of q that is not
// finite is all NaN.
#pragma once

#include "mx_common.h"
#include "mx_internal.h"

namespace q4k {

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr float kMinusInf = -__builtin_inff();
// What the weights' exponents are counted from for a largest x of mx, and how far
// above it x may come.  From 2^24 on fp32 has no such steps, and mx itself is taken.
constexpr float kMostExponent = 14.0f;
__device__ __forceinline__ float exponent_base(float mx) {
  return __builtin_fabsf(mx) < 0x1p24f ? mx - 10.0f : mx;
}
// The power that the largest code takes within fp16: 448 * 2^6, 6 * 2^13.
template <int FMT> constexpr int kCodeExponent = FMT == MX_FP8 ? 6 : 13;

// Keys lo .. hi (none where hi < lo).
struct Range { int lo, hi; };

struct Sequence {
  int q0, nq, total, nk;  // first token, rows' tokens, all of its tokens, keys
  __device__ __forceinline__ Range sees(const AttentionArgs &a, int i) const {
    const int hi = a.causal ? nk - total + i : nk - 1;
    return {a.window ? max(0, hi - a.window + 1) : 0, hi};
  }
};

// Each share of keys has at least so many.
constexpr int kMinKeys = 128;

// Starts and counts as they should be, whatever they hold.
__device__ __forceinline__ Sequence sequence_of(const AttentionArgs &a, int s) {
  Sequence r;
  r.q0 = min(max(a.starts[s], 0), a.n_tokens);
  r.total = min(max(a.starts[s + 1], r.q0), a.n_tokens) - r.q0;
  r.nq = min(r.total, a.max_queries);
  r.nk = min(max(a.counts[s], 0), a.pages_per_seq * a.page_size);
  return r;
}

__device__ __forceinline__ uint32_t swap_max_u32(uint32_t v) {  // over lanes 16 and 32 apart
  const auto x = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  const uint32_t x0 = x[0], x1 = x[1];
  v = max(x0, x1);
  const auto y = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  const uint32_t y0 = y[0], y1 = y[1];
  return max(y0, y1);
}

// Sums over the lanes up to each: within rows of 16, then the rows' last ones.
template <int CTRL, int ROWS> __device__ __forceinline__ uint32_t add_dpp(uint32_t v) {
  return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v = add_dpp<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
  v = add_dpp<0x112, 0xF>(v);
  v = add_dpp<0x114, 0xF>(v);
  v = add_dpp<0x118, 0xF>(v);
  v = add_dpp<0x142, 0xA>(v);  // row_bcast 15, 31
  return add_dpp<0x143, 0xC>(v);
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// What one workgroup works on, in steps of KEYS keys: rows r0 .. of a
// sequence's (token, head of the group) pairs and the steps of keys that any of
// them sees, or its share.  A unit is such a share, for all key heads.
struct Work {
  Sequence seq;
  int index, kv_head, r0, rows, split, splits;  // index of the sequence; splits: shares in use
  uint32_t unit;   // of share 0
  Range any, all;  // keys that one row at least sees, that all do
  int begin, first, last;  // key of step 0; this share's steps
};

// The sequences' units lie one after the other: a sequence of `tiles` tiles whose
// keys make `shares` shares at most has tiles * shares.  The shares' length is one
// for the whole batch, so that about a.shares_wanted workgroups come out and none
// works longer than that; a tile's last share is what is left, often much less, and
// a window's tiles see fewer keys (their own tokens') than are counted here (those of
// max_queries).  Every wave finds its place for itself, 64 sequences at a time.
// BY_TILE: `n` counts tiles, not units.
template <int ROWS, int KEYS, bool BY_TILE>
__device__ __forceinline__ bool find_work(const AttentionArgs &a, uint32_t n, Work &w, int &tile,
                                          int &share) {
  const int lane = threadIdx.x & 63;
  const auto sizes = [&](int s, Sequence &q, uint32_t &tiles, uint32_t &steps) {
    tiles = steps = 0;
    if (s >= a.n_seqs) return;
    q = sequence_of(a, s);
    tiles = (q.nq * a.group + ROWS - 1) / ROWS;
    const int most = a.window ? (int)min((int64_t)q.nk, (int64_t)a.window + a.max_queries + KEYS) : q.nk;
    steps = (most + KEYS - 1) / KEYS;
  };
  Sequence q;
  uint32_t tiles, steps, total = 0;
  share = 0x7FFFFFFF;
  if (a.shares_wanted > 0) {
    for (int s = lane; s - lane < a.n_seqs; s += 64) {
      sizes(s, q, tiles, steps);
      total += lane_value(wave_scan(tiles * steps), 63);
    }
    share = max((int)(total / a.shares_wanted) + 1, kMinKeys / KEYS);
  }
  uint32_t units_before = 0, tiles_before = 0;
  for (int s = lane; s - lane < a.n_seqs; s += 64) {
    sizes(s, q, tiles, steps);
    const uint32_t shares = a.shares_wanted > 0 ? max(1u, (steps + share - 1) / share) : 1;
    const uint32_t units_to = units_before + wave_scan(tiles * shares);
    const uint32_t tiles_to = BY_TILE ? tiles_before + wave_scan(tiles) : 0;
    const uint64_t after = __builtin_amdgcn_ballot_w64((BY_TILE ? tiles_to : units_to) > n);
    if (after != 0) {
      const int at = __builtin_ctzll(after);
      const uint32_t mine_shares = lane_value(shares, at), mine_tiles = lane_value(tiles, at);
      const uint32_t first = lane_value(units_to, at) - mine_tiles * mine_shares;
      if constexpr (BY_TILE) {
        tile = n - (lane_value(tiles_to, at) - mine_tiles);
        w.split = 0;
      } else {
        tile = (n - first) / mine_shares;
        w.split = (n - first) - tile * mine_shares;
      }
      w.unit = first + tile * mine_shares;
      tile = mine_tiles - 1 - tile;  // those with most keys first
      w.index = s - lane + at;
      w.seq.q0 = lane_value(q.q0, at);
      w.seq.nq = lane_value(q.nq, at);
      w.seq.total = lane_value(q.total, at);
      w.seq.nk = lane_value(q.nk, at);
      return true;
    }
    units_before = lane_value(units_to, 63);
    if (BY_TILE) tiles_before = lane_value(tiles_to, 63);
  }
  return false;
}

// The work of a block; blocks count units (tiles) of all key heads, the heads of
// one next to each other.
template <int ROWS, int KEYS, bool BY_TILE = false>
__device__ __forceinline__ bool work_of(const AttentionArgs &a, uint32_t block, Work &w) {
  const uint32_t n = a.by_kv_heads.of(block);
  w.kv_head = block - n * a.n_kv_heads;
  int tile, share = 0x7FFFFFFF;
  if (a.planned) {
    if (!find_work<ROWS, KEYS, BY_TILE>(a, n, w, tile, share)) return false;
  } else {  // too many sequences to look through: as many tiles as the longest may have
    w.index = a.by_tiles.of(n);
    tile = a.tiles - 1 - (n - w.index * a.tiles);
    w.split = 0;
    w.unit = n;
    w.seq = sequence_of(a, w.index);
  }
  w.r0 = tile * ROWS;
  const int all_rows = w.seq.nq * a.group;
  if (w.r0 >= all_rows) return false;
  w.rows = min(ROWS, all_rows - w.r0);
  const Range one = w.seq.sees(a, a.by_group.of(w.r0));
  const Range two = w.seq.sees(a, a.by_group.of(w.r0 + w.rows - 1));
  w.any = {one.lo, two.hi};
  w.all = {two.lo, one.hi};
  w.begin = w.any.lo & ~(KEYS - 1);
  const int steps = w.any.hi < w.any.lo ? 0 : (w.any.hi + KEYS - w.begin) / KEYS;
  share = min(share, max(steps, 1));
  w.splits = max(1, (steps + share - 1) / share);
  w.first = w.split * share;
  w.last = min(steps, w.first + share);
  return w.split < w.splits;
}

// Where a row of a share has its part: rows, then rows' largest x and sums.
template <int ROWS>
__device__ __forceinline__ int64_t part_row(const AttentionArgs &a, const Work &w, int share, int row) {
  return ((int64_t)(w.unit + share) * a.n_kv_heads + w.kv_head) * ROWS + row;
}
__device__ __forceinline__ float2 *part_stats(const AttentionArgs &a) {
  return reinterpret_cast<float2 *>(a.partial + a.n_parts * a.head_dim);
}

__device__ __forceinline__ float swap_max16(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto h = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t x = h[0], y = h[1];
  return fmaxf(__uint_as_float(x), __uint_as_float(y));
}
__device__ __forceinline__ float swap_max32(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t x = h[0], y = h[1];
  return fmaxf(__uint_as_float(x), __uint_as_float(y));
}

__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}
// Maxima of the two 16-bit halves over the wave, as a scalar.
__device__ __forceinline__ uint32_t wave_pk_max(uint32_t v) {
  v = pk_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
  v = pk_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
  v = pk_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));
  v = pk_max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));
  const auto h = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  const uint32_t h0 = h[0], h1 = h[1];
  v = pk_max(h0, h1);
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  const uint32_t r0 = r[0], r1 = r[1];
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)pk_max(r0, r1));
}

// A scale byte's part in a reference: NaN blocks take none.
__device__ __forceinline__ uint32_t scale_rank(uint32_t s) { return s == 255 ? 0 : s; }
// 2^(s - ref + kCodeExponent) as the conversions take it; base = 127 + kCodeExponent - ref.
__device__ __forceinline__ float block_scale(uint32_t s, int base) {
  const int e = min(max((int)s + base, 0), 254);
  return __builtin_bit_cast(float, s == 255 ? 0x7FC00000u : (uint32_t)e << 23);
}

// A reference: that of the keys taken together, or the one before as long as it
// is no lower and at most 2^8 above, so that it seldom changes.  What is summed up
// carries the values'.  It may fall as well: a single large value takes no bits
// from those of other keys.  Not below 64, so that keys and values below 2^-55 lose
// bits.
constexpr int kFirstRef = 127, kLastRef = 64;
__device__ __forceinline__ int reference(int before, int top) {
  const int now = max(top, kLastRef);
  return now > before || now + 8 < before ? now : before;
}

// Values without a reference may lie this far above that of the sums, which is raised
// if they do not: a sum of them stays below 2^120.
constexpr int kMixedShift = 8, kMixedReach = 60;

// Under one reference a sum is below 2^60 (2^44 of weights, 2^16 of codes), but what
// was summed under a higher one grows by the fall, up to 2^190 of it.  Where a row's
// largest sum, of magnitude bits `top`, would pass 2^126, this power of two is held
// back: sums and sum of weights are smaller by it, and so are the weights until the
// reference or the maximum changes again, which count for less than 2^-65 of what
// there is.
__device__ __forceinline__ int held_back(uint32_t top, int fall) {
  return max(0, (int)(top >> 23) + fall - 252);
}
// A sum's magnitude bits; what is not finite stays so, and holds nothing back.
__device__ __forceinline__ uint32_t sum_bits(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
  return b >= 0x7F800000u ? 0 : b;
}

// Eight codes (two dwords of e4m3, one of e2m1) as a matrix operand.
template <int FMT> __device__ __forceinline__ half8_t codes_operand(const uint32_t *c, float scale) {
  half2_t h0, h1, h2, h3;
  if constexpr (FMT == MX_FP8) {
    h0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)c[0], scale, 0);
    h1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)c[0], scale, 1);
    h2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)c[1], scale, 0);
    h3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)c[1], scale, 1);
  } else {
    h0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c[0], scale, 0);
    h1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c[0], scale, 1);
    h2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c[0], scale, 2);
    h3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c[0], scale, 3);
  }
  return half8_t{h0.x, h0.y, h1.x, h1.y, h2.x, h2.y, h3.x, h3.y};
}

template <int W> __device__ __forceinline__ void load_codes(const uint8_t *p, uint32_t (&c)[W]) {
  if constexpr (W == 4) {
    const u32x4 v = *reinterpret_cast<const u32x4 *>(p);
    c[0] = v[0]; c[1] = v[1]; c[2] = v[2]; c[3] = v[3];
  } else {
    const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
    c[0] = v[0]; c[1] = v[1];
  }
}

// The scale bytes of a lane's blocks 2 p + g / 2 of a row: as loaded (FOURS:
// whole dwords of four blocks, for rows made of them; else bytes), and, once
// settled, two to a dword.  Both ways in one kernel, by a branch, would be waited
// for where the branches meet, and so would all loads before them.
struct __attribute__((packed)) Packed4 { uint32_t v; };  // at any alignment
template <int ND, bool FOURS> struct RawScales {
  static constexpr int S = (ND + 1) / 2;
  uint32_t raw[FOURS ? S : ND], pair[S];
  __device__ __forceinline__ void load(const uint8_t *row, int nb, int g) {
#pragma unroll
    for (int i = 0; i < (FOURS ? S : ND); i++) {
      if constexpr (FOURS) raw[i] = reinterpret_cast<const Packed4 *>(row + 4 * i)->v;
      else raw[i] = row[min(2 * i + (g >> 1), nb - 1)];
    }
  }
  __device__ __forceinline__ void settle(int g) {
#pragma unroll
    for (int i = 0; i < S; i++) {
      if constexpr (FOURS) pair[i] = raw[i] >> (8 * (g >> 1)) & 0x00FF00FFu;
      else pair[i] = raw[2 * i] | (2 * i + 1 < ND ? raw[2 * i + 1 < ND ? 2 * i + 1 : 0] << 16 : 0);
    }
  }
  // 2^(s + base - 127), s + base <= 254; NaN blocks as any others
  __device__ __forceinline__ void powers(int base, float (&f)[ND]) const {
    const i16x2 add = {(short)base, (short)base}, none = {0, 0};
#pragma unroll
    for (int i = 0; i < S; i++) {
      const uint32_t e = __builtin_bit_cast(
          uint32_t, __builtin_elementwise_max(__builtin_bit_cast(i16x2, pair[i]) + add, none));
      f[2 * i] = __builtin_bit_cast(float, e << 23);
      if (2 * i + 1 < ND) f[2 * i + 1 < ND ? 2 * i + 1 : 0] = __builtin_bit_cast(float, (e & 0xFFFF0000u) << 7);
    }
  }
  __device__ __forceinline__ void clear(int p) { pair[p / 2] &= p & 1 ? 0x0000FFFFu : 0xFFFF0000u; }
  __device__ __forceinline__ uint32_t of(int p) const { return pair[p / 2] >> (16 * (p & 1)) & 0xFFFF; }
};

template <int FMT>
__device__ __forceinline__ bf16x8 codes_operand_bf16(const uint32_t *c, float scale) {
  bf16x2 h0, h1, h2, h3;
  if constexpr (FMT == MX_FP8) {
    h0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[0], scale, 0);
    h1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[0], scale, 1);
    h2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[1], scale, 0);
    h3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[1], scale, 1);
  } else {
    h0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[0], scale, 0);
    h1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[0], scale, 1);
    h2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[0], scale, 2);
    h3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[0], scale, 3);
  }
  return bf16x8{h0.x, h0.y, h1.x, h1.y, h2.x, h2.y, h3.x, h3.y};
}

// Whether 16 codes or their scale hold a NaN.
template <int FMT, int W>
__device__ __forceinline__ bool has_nan(const uint32_t (&c)[W], uint32_t s) {
  bool r = s == 255;
  if constexpr (FMT == MX_FP8)
#pragma unroll
    for (int i = 0; i < W; i++) r |= (((c[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
  return r;
}

// What a row's scores are multiplied by: 2^power of a.scale, and no infinity (0
// times it is no score; others are beyond fp32 with it or without).
__device__ __forceinline__ float score_scale(float scale, int power) {
  return __builtin_ldexpf(scale, min(power, 127));
}

// Eight consecutive values of a row of q, as they lie in memory and in fp32: NP
// = 2 stands for fp32, one operand for the 16-bit types.  No branch lies
// between loads, so that all are on their way together.
template <int NP> struct RawQ { Raw8<NP == 2 ? MX_F32 : MX_F16> v; };
template <int NP> __device__ __forceinline__ RawQ<NP> load_q8(const AttentionArgs &a, int64_t at) {
  return {load_raw8<NP == 2 ? MX_F32 : MX_F16>(static_cast<const uint8_t *>(a.q) + at * (2 * NP), 0)};
}
template <int NP>
__device__ __forceinline__ void q8_to_f32(const AttentionArgs &a, const RawQ<NP> &r, float (&f)[8]) {
  if constexpr (NP == 2) {
    raw8_to_f32<MX_F32>(r.v, f);
  } else if (a.type == MX_BF16) {
    raw8_to_f32<MX_BF16>({r.v.v}, f);
  } else {
    raw8_to_f32<MX_F16>(r.v, f);
  }
}

__device__ __forceinline__ void store_y4(const AttentionArgs &a, int64_t at, f32x4 v) {
  if (a.type == MX_F32) {
    *reinterpret_cast<f32x4 *>(static_cast<float *>(a.y) + at) = v;
  } else {
    u32x2 r;
    if (a.type == MX_BF16) {
      r[0] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[0], (__bf16)v[1]});
      r[1] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2], (__bf16)v[3]});
    } else {
      r[0] = as_u32h(half2_t{(_Float16)v[0], (_Float16)v[1]});
      r[1] = as_u32h(half2_t{(_Float16)v[2], (_Float16)v[3]});
    }
    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.y) + at) = r;
  }
}

// The exponent e of a row whose largest magnitude has these bits (0 for a row of zeros).
__device__ __forceinline__ int row_exponent(uint32_t amax_bits) {
  return amax_bits == 0 ? 0 : (int)(amax_bits >> 23) - 127 - 14;
}

// The share of a partial result whose weights count from m in one whose do from most.  A
// part without keys has m = -inf and zeros; one whose x are all NaN has m =
// -inf and NaNs, which have to stay.
__device__ __forceinline__ float part_share(float m, float most) {
  return m == kMinusInf ? 1.0f : __builtin_amdgcn_exp2f(m - most);
}

// Before a row's sums are divided by those of its weights they are up to 2^44
// (2^14 for each of 2^30 keys) times the largest value, which alone may be next to
// fp32's largest: they are kept times 2^-44, and the quotient is put back.
constexpr int kSumExponent = 44;
__device__ __forceinline__ f32x4 quotient(f32x4 v, float sum) {
  v *= sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = __builtin_ldexpf(v[i], kSumExponent);
  return v;
}

// 128 rows a workgroup, 64 keys a step.
constexpr int kTiledRows = 128, kTiledKeys = 64;
hipError_t attention_tiled_launch(const AttentionArgs &a, int blocks, hipStream_t stream);

}  // namespace q4k
