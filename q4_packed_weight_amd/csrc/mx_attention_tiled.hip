// mx_attention_tiled.hip -- attention over a paged MX cache for many rows:
// chunks of new tokens, 32 rows a wave.
#include <type_traits>

#include "mx_attention.h"

namespace q4k {
namespace {

constexpr int kWaves = 4;
constexpr int kRows = kTiledRows;
constexpr int kTile = kTiledKeys;
static_assert(kRows == 32 * kWaves, "32 rows a wave");
constexpr int kWaveKeys = kTile / kWaves;  // that a wave stages: 16, one step of V^T P^T
typedef float f32x16 __attribute__((ext_vector_type(16)));

// What a wave says of the 16 keys it has staged: a scale above its reference,
// one at most 2^8 below it, a page that is none; of mixed tiles a NaN value and,
// in the byte above, the values' largest scale.
enum : uint32_t { kOver = 1, kNearK = 2, kNearV = 4, kAbsent = 8, kNan = 16 };
constexpr int kNoKey = 0x7FFF;  // in place of a key's power

// A wave's share of a tile as it lies in memory: 16 codes (dims 16 n .. of lane
// n of a key's LP lanes) in each pass.
template <int FMT, int ND> struct TileData {
  static constexpr int LP = ND == 1 ? 4 : ND == 2 ? 8 : 16;
  static constexpr int PASSES = kWaveKeys * LP / 64;
  static constexpr int W = FMT == MX_FP8 ? 4 : 2;
  uint32_t k[PASSES][W], v[PASSES][W];
  uint8_t ks[PASSES], vs[PASSES];
  bool ok[PASSES];  // a key that some row sees, in a page that there is
};

// A copy that the compiler does not see through.
__device__ __forceinline__ int in_place(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

template <int LP> __device__ __forceinline__ uint32_t max_of_key(uint32_t v) {
  v = max_dpp_step<0xB1>(v);
  v = max_dpp_step<0x4E>(v);
  if constexpr (LP >= 8) v = max_dpp_step<0x141>(v);
  if constexpr (LP >= 16) v = max_dpp_step<0x140>(v);
  return v;
}

// As in the form for few rows, scores are S^T = K Q^T and the sums O^T += V^T P^T,
// here of 32 keys by 32 rows: a row's statistics are two lanes' own, and sixteen of
// a lane's weights are two operands as they stand.  The four waves stage a tile of
// 64 keys once for their 128 rows, 16 keys each, converted on the way into LDS (a
// conversion of two codes a lane is one instruction, and each is made once instead
// of by every wave); two tiles in LDS and one in registers, two workgroups a CU.
// The tile's references are those of the tiles before as long as they hold (stage
// says so, stage_again mends it), so that nothing is exchanged before the barrier.
// Bound by the waits of two waves a SIMD: of 2048 tokens over 8192 keys (32 heads of
// 128, 241 GFLOP, 330 to 348 us by the card, 0.7 PFLOP/s, half of a large fp16
// product's rate) the matrix pipe works 28% and the vector unit 44% of the time.
// Tried, when it took 322: operands read ahead in a fixed order, with the sums kept in
// memory around that loop so that its registers suffice 361 us, without 390; 2 x 32-key
// halves 477.
// WHOLE: pages of a multiple of 16 keys, so that a wave's 16 lie in one and
// their addresses are scalars (351 against 341 us when it came).
template <int NP, int FMT, int ND, bool WHOLE>
__global__ __launch_bounds__(kWaves * 64, ND <= 2 ? 2 : 1) void attention_tiled_kernel(AttentionArgs a) {
  constexpr int DP = 64 * ND;
  constexpr int KS = 2 * DP + 16, VS = 2 * DP + 64;  // bytes of a key's row in LDS, over all banks
  constexpr int X = kCodeExponent<FMT>;
  typedef TileData<FMT, ND> Data;
  constexpr int LP = Data::LP, PASSES = Data::PASSES, W = Data::W;
  __shared__ __attribute__((aligned(16))) uint8_t k_lds[2][kTile * KS];
  __shared__ __attribute__((aligned(16))) uint8_t v_lds[2][kTile * VS];
  __shared__ __attribute__((aligned(16))) int powers[2][kTile];
  __shared__ __attribute__((aligned(16))) uint32_t staged[2][kWaves], tops[kWaves];
  __shared__ float2 held[kWaves][32];  // where any_held: rows' m without what is held back, and that
  Work w;
  if (!work_of<kRows, kTile>(a, blockIdx.x, w)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r32 = lane & 31, half = lane >> 5;
  const int D = a.head_dim, nb = D / 32;
  const int64_t code_row = FMT == MX_FP8 ? D : D / 2;

  // queries: dims 16 s + 8 half .. + 7 in step s; rows behind the last are its copies
  const bool active = 32 * wave < w.rows;
  const int last_row = w.r0 + w.rows - 1;
  const int row = min(w.r0 + 32 * wave + r32, last_row);
  const int token = a.by_group.of(row);
  const Range mine = w.seq.sees(a, token);
  const Range one = w.seq.sees(a, a.by_group.of(min(w.r0 + 32 * wave, last_row)));
  const Range two = w.seq.sees(a, a.by_group.of(min(w.r0 + 32 * wave + 31, last_row)));
  half8_t q[NP][DP / 16];
  int row_power;
  // the largest x is the largest score: a negative scale's sign goes to q
  const float scale = __builtin_fabsf(a.scale);
  {
    const int64_t at = (int64_t)(w.seq.q0 + token) * a.q_stride +
                       (int64_t)(w.kv_head * a.group + row - token * a.group) * D + 8 * half;
    RawQ<NP> raw[DP / 16];
#pragma unroll
    for (int s = 0; s < DP / 16; s++) raw[s] = load_q8<NP>(a, at + (16 * s < D ? 16 * s : 0));
    float f[DP / 16][8];
    uint32_t amax = 0;
#pragma unroll
    for (int s = 0; s < DP / 16; s++) {
      q8_to_f32<NP>(a, raw[s], f[s]);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        if (16 * s >= D) f[s][i] = 0.0f;
        const uint32_t b = __builtin_bit_cast(uint32_t, f[s][i]) & 0x7FFFFFFFu;
        amax = b > amax ? b : amax;
      }
    }
    const auto y = __builtin_amdgcn_permlane32_swap(amax, amax, false, false);
    const uint32_t y0 = y[0], y1 = y[1];
    amax = max(y0, y1);
    const int e = row_exponent(amax);
    const float sign = amax >= 0x7F800000u ? __builtin_nanf("") : a.scale < 0.0f ? -1.0f : 1.0f;
    row_power = e + a.scale_power;
#pragma unroll
    for (int s = 0; s < DP / 16; s++)
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float v = __builtin_ldexpf(f[s][i] * sign, -e);
        q[0][s][i] = (_Float16)v;
        if constexpr (NP == 2) q[1][s][i] = (_Float16)(v - (float)q[0][s][i]);
      }
  }

  const int32_t *const table = a.table + (int64_t)w.index * a.pages_per_seq;
  // Key of a wave's pass and 16 dims of it; lanes behind head_dim do what the
  // key's first lane does, and the keys' columns there are zeros once and for all.
  const int lane_key = lane / LP, sub = 16 * (lane & (LP - 1)) < D ? lane & (LP - 1) : 0;
  if (D != DP) {
    const int pad = (DP - D) / 8;
    for (int i = threadIdx.x; i < 2 * kTile * pad; i += kWaves * 64)
      *reinterpret_cast<u32x4 *>(k_lds[0] + i / pad * KS + 2 * D + 16 * (i % pad)) = u32x4{0, 0, 0, 0};
  }
  // Pages of the keys, then their codes: every lane loads, absent keys a row that
  // there is, without a branch; stage puts zeros there.
  Data d;
  int pages[WHOLE ? 1 : PASSES];
  const auto key_of = [&](int t, int p) __attribute__((always_inline)) {
    return w.begin + t * kTile + kWaveKeys * wave + (WHOLE ? 0 : 64 / LP * p + lane_key);
  };
  // The compiler must not know that one page is the same for all lanes, or it waits
  // for it, and so for all loads before it, at once, to have it in a scalar.
  const int of_lane = in_place(0);
  const auto load_pages = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < (WHOLE ? 1 : PASSES); p++)
      pages[p] = table[a.by_page.of(min(max(key_of(t, p), w.any.lo), w.any.hi)) + (WHOLE ? of_lane : 0)];
  };
  const uint32_t lane_code = (WHOLE ? lane_key * (int)code_row : 0) +
                             16 * sub * (FMT == MX_FP8 ? 2 : 1) / 2;
  const uint32_t lane_scale = (WHOLE ? lane_key * nb : 0) + (sub >> 1);
  const auto load = [&](int t) __attribute__((always_inline)) {
    const uint8_t *k, *v, *ks, *vs;
#pragma unroll
    for (int p = 0; p < PASSES; p++) {
      if (!WHOLE || p == 0) {
        const int key = key_of(t, p);
        const int page = WHOLE ? __builtin_amdgcn_readfirstlane(pages[p]) : pages[p];
        d.ok[p] = t < w.last && (uint32_t)page < (uint32_t)a.n_pages && (WHOLE || (key >= w.any.lo && key <= w.any.hi));
        const uint32_t place = key - a.by_page.of(key) * a.page_size;
        const uint32_t r = d.ok[p] ? (page * a.n_kv_heads + w.kv_head) * a.page_size + place : 0;
        const uint64_t c = (uint64_t)r * code_row, s = (uint64_t)r * nb;
        k = a.k_codes + c, v = a.v_codes + c, ks = a.k_scales + s, vs = a.v_scales + s;
      }
      const uint32_t c = lane_code + (WHOLE ? 64 / LP * p * (int)code_row : 0);
      const uint32_t s = lane_scale + (WHOLE ? 64 / LP * p * nb : 0);
      load_codes(k + c, d.k[p]);
      load_codes(v + c, d.v[p]);
      d.ks[p] = ks[s];
      d.vs[p] = vs[s];
    }
  };
  // keys that some rows see and others do not, or none
  const auto is_mixed = [&](int t) __attribute__((always_inline)) {
    const int first = w.begin + t * kTile;
    return first < w.all.lo || first + kTile - 1 > w.all.hi;
  };
  int k_ref = kFirstRef, v_ref = kFirstRef;

  // The tile's share into LDS as fp16 under the references (mixed: keys under
  // their own, values as bf16).
  const auto stage = [&](int t, bool mixed) __attribute__((always_inline)) {
    const int b = t & 1;
    bool absent = false, nan = false;
    uint32_t k_top = 0, v_top = 0;
    if constexpr (WHOLE) {
      absent = !d.ok[0];
#pragma unroll
      for (int p = 1; p < PASSES; p++) d.ok[p] = d.ok[0];
      if (mixed) {
#pragma unroll
        for (int p = 0; p < PASSES; p++) {
          const int key = key_of(t, 0) + 64 / LP * p + lane_key;
          d.ok[p] = d.ok[p] && key >= w.any.lo && key <= w.any.hi;
          absent |= !d.ok[p];
        }
      }
    } else {
#pragma unroll
      for (int p = 0; p < PASSES; p++) absent |= !d.ok[p];
    }
    absent = __builtin_amdgcn_ballot_w64(absent) != 0;
    if (absent) {
#pragma unroll
      for (int p = 0; p < PASSES; p++) {
        if (!d.ok[p]) {
#pragma unroll
          for (int i = 0; i < W; i++) d.k[p][i] = d.v[p][i] = 0;
          d.ks[p] = d.vs[p] = 0;
        }
      }
    }
#pragma unroll
    for (int p = 0; p < PASSES; p++) {
      const int n = kWaveKeys * wave + 64 / LP * p + lane_key;
      uint8_t *const k_to = k_lds[b] + n * KS + 32 * sub, *const v_to = v_lds[b] + n * VS + 32 * sub;
      int k_base = 127 + X - k_ref;
      if (mixed) {
        const int own = (int)max_of_key<LP>(scale_rank(d.ks[p]));
        k_base = 127 + X - own;
        nan |= has_nan<FMT>(d.v[p], d.vs[p]);
        v_top = max(v_top, scale_rank(d.vs[p]));
        if (sub == 0) powers[b][n] = d.ok[p] ? own - X - 127 : kNoKey;
        const float s = block_scale(d.vs[p], -kMixedShift);
        *reinterpret_cast<bf16x8 *>(v_to) = codes_operand_bf16<FMT>(&d.v[p][0], s);
        *reinterpret_cast<bf16x8 *>(v_to + 16) = codes_operand_bf16<FMT>(&d.v[p][W / 2], s);
      } else {
        k_top = max(k_top, scale_rank(d.ks[p]));
        v_top = max(v_top, scale_rank(d.vs[p]));
        const float s = block_scale(d.vs[p], 127 + X - v_ref);
        *reinterpret_cast<half8_t *>(v_to) = codes_operand<FMT>(&d.v[p][0], s);
        *reinterpret_cast<half8_t *>(v_to + 16) = codes_operand<FMT>(&d.v[p][W / 2], s);
      }
      const float s = block_scale(d.ks[p], k_base);
      *reinterpret_cast<half8_t *>(k_to) = codes_operand<FMT>(&d.k[p][0], s);
      *reinterpret_cast<half8_t *>(k_to + 16) = codes_operand<FMT>(&d.k[p][W / 2], s);
    }
    uint32_t word = 0;
    if (mixed) {
      word = wave_pk_max(v_top) << 8 | (__builtin_amdgcn_ballot_w64(nan) != 0 ? kNan : 0);
    } else {
      if (__builtin_amdgcn_ballot_w64((int)k_top > k_ref || (int)v_top > v_ref) != 0) word |= kOver;
      if (k_ref == kLastRef || __builtin_amdgcn_ballot_w64((int)k_top + 8 >= k_ref) != 0) word |= kNearK;
      if (v_ref == kLastRef || __builtin_amdgcn_ballot_w64((int)v_top + 8 >= v_ref) != 0) word |= kNearV;
      if (absent) word |= kAbsent;
    }
    if (lane == 0) staged[b][wave] = word;
  };
  // The same without a branch, for keys that are all there and all seen; a NaN
  // block counts as a scale above the reference.
  const int to_key = kWaveKeys * wave + lane_key;
  const auto stage_fast = [&](int b) __attribute__((always_inline)) {
    uint32_t k_top = 0, v_top = 0;
    uint8_t *const k_to = k_lds[b] + to_key * KS + 32 * sub, *const v_to = v_lds[b] + to_key * VS + 32 * sub;
    const int k_base = 127 + X - k_ref, v_base = 127 + X - v_ref;
#pragma unroll
    for (int p = 0; p < PASSES; p++) {
      const float f = __builtin_bit_cast(float, (uint32_t)(max((int)d.ks[p], -k_base) + k_base) << 23);
      const float g = __builtin_bit_cast(float, (uint32_t)(max((int)d.vs[p], -v_base) + v_base) << 23);
      k_top = max(k_top, (uint32_t)d.ks[p]);
      v_top = max(v_top, (uint32_t)d.vs[p]);
      *reinterpret_cast<half8_t *>(k_to + 64 / LP * p * KS) = codes_operand<FMT>(&d.k[p][0], f);
      *reinterpret_cast<half8_t *>(k_to + 64 / LP * p * KS + 16) = codes_operand<FMT>(&d.k[p][W / 2], f);
      *reinterpret_cast<half8_t *>(v_to + 64 / LP * p * VS) = codes_operand<FMT>(&d.v[p][0], g);
      *reinterpret_cast<half8_t *>(v_to + 64 / LP * p * VS + 16) = codes_operand<FMT>(&d.v[p][W / 2], g);
    }
    uint32_t word = 0;
    word |= __builtin_amdgcn_ballot_w64((int)k_top > k_ref || (int)v_top > v_ref) != 0 ? kOver : 0;
    word |= k_ref == kLastRef || __builtin_amdgcn_ballot_w64((int)k_top + 8 >= k_ref) != 0 ? kNearK : 0;
    word |= v_ref == kLastRef || __builtin_amdgcn_ballot_w64((int)v_top + 8 >= v_ref) != 0 ? kNearV : 0;
    staged[b][wave] = word;  // by all lanes
  };

  f32x16 acc[2 * ND];
#pragma unroll
  for (int t = 0; t < 2 * ND; t++)
#pragma unroll
    for (int i = 0; i < 16; i++) acc[t][i] = 0.0f;
  float m = kMinusInf, l = 0.0f;
  bool any_held = false;
  typedef __attribute__((address_space(3))) s16x4 LdsS16x4;
  const int v_at = (4 * half + (lane >> 2 & 3)) * VS + 32 * (lane >> 4 & 1) + 8 * (lane & 3);
  const int k_at = r32 * KS + 16 * half;

  // 32 dims of the 16 keys of step n, transposed: keys 4 half .. + 3 and 8 + 4 half .. + 3
  const auto value_operand = [&](int b, int n, int t) __attribute__((always_inline)) {
    const uint8_t *const at = v_lds[b] + v_at + 16 * n * VS + 64 * t;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4 *)at);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4 *)(at + 8 * VS));
    return s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  const auto scores = [&](int b, f32x16 (&s)[2]) __attribute__((always_inline)) {
    const f32x16 zeros = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int n = 0; n < DP / 16; n++) {
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const half8_t k = *reinterpret_cast<const half8_t *>(k_lds[b] + k_at + 32 * j * KS + 32 * n);
#pragma unroll
        for (int p = 0; p < NP; p++)
          s[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[p][n], n + p == 0 ? zeros : s[j], 0, 0, 0);
      }
    }
  };
  // what was summed to the values' new reference
  const auto refer = [&](int v_new) __attribute__((always_inline)) {
    int power = v_ref - v_new;
    if (power > 0 || any_held) {
      float2 kept = make_float2(m, 0.0f);
      if (any_held) kept = held[wave][r32];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 32 * ND; i++) top = max(top, sum_bits(acc[i >> 4][i & 15]));
      const auto y = __builtin_amdgcn_permlane32_swap(top, top, false, false);
      const uint32_t y0 = y[0], y1 = y[1];
      power += (int)kept.y;
      const int more = held_back(max(y0, y1), power);
      power -= more;
      l = __builtin_ldexpf(l, (int)kept.y - more);
      m = kept.x + more;
      any_held = __builtin_amdgcn_ballot_w64(more != 0) != 0;
      if (any_held) held[wave][r32] = make_float2(kept.x, more);
    }
#pragma unroll
    for (int i = 0; i < 32 * ND; i++) acc[i >> 4][i & 15] = __builtin_ldexpf(acc[i >> 4][i & 15], power);
    v_ref = v_new;
  };
  // as in the form for few rows: a maximum up to 2^4 too low stays
  const auto raise = [&](float mx) __attribute__((always_inline)) {
    mx = swap_max32(mx);
    const bool up = mx - m > kMostExponent;
    if (__builtin_amdgcn_ballot_w64(up) != 0) {
      const float to = up ? exponent_base(mx) : m, f = up ? __builtin_amdgcn_exp2f(m - to) : 1.0f;
      l *= f;
#pragma unroll
      for (int t = 0; t < 2 * ND; t++)
#pragma unroll
        for (int i = 0; i < 16; i++) acc[t][i] *= f;
      m = to;
      if (any_held && up) held[wave][r32] = make_float2(m, 0.0f);
    }
    return m == kMinusInf ? 0.0f : m;
  };

  // AND_NEXT: the next tile is staged among the scores' products
  const auto compute = [&](int b, auto and_next) __attribute__((always_inline)) {
    f32x16 s[2];
    scores(b, s);
    if constexpr (decltype(and_next)::value) stage_fast(b ^ 1);
    float c = score_scale(scale, row_power + k_ref - X - 127);
    float mx = s[0][0];
#pragma unroll
    for (int i = 1; i < 32; i++) mx = fmaxf(mx, s[i >> 4][i & 15]);
    // x - m by one rounding is off by what m was rounded by, which is no matter while it
    // is a small part of one; beyond, both are rounded alike
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(__builtin_fabsf(mx * c) >= 0x1p23f) != 0, 0)) {
#pragma clang fp contract(off)
#pragma unroll
      for (int i = 0; i < 32; i++) s[i >> 4][i & 15] *= c;
      mx *= c;
      c = 1.0f;
    }
    const float less = raise(mx * c);
#pragma unroll
    for (int n = 0; n < kWaves; n++) {
      half8_t p[NP];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n >> 1][8 * (n & 1) + i], c, -less));
        l += e;
        p[0][i] = (_Float16)e;
        if constexpr (NP == 2) p[1][i] = (_Float16)(e - (float)p[0][i]);
      }
#pragma unroll
      for (int t = 0; t < 2 * ND; t++) {
        const half8_t v = __builtin_bit_cast(half8_t, value_operand(b, n, t));
#pragma unroll
        for (int k = 0; k < NP; k++)
          acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p[k], acc[t], 0, 0, 0);
      }
    }
  };

  const auto compute_mixed = [&](int b, int first, bool nans) __attribute__((always_inline)) {
    f32x16 s[2];
    scores(b, s);
    uint32_t sees = 0;
    float mx = kMinusInf;
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int at = 32 * j + 2 * i + 4 * half;
        const i32x4 c = *reinterpret_cast<const i32x4 *>(&powers[b][at]);
#pragma unroll
        for (int n = 0; n < 4; n++) {
          const int key = first + at + n;
          const bool see = c[n] != kNoKey && key >= mine.lo && key <= mine.hi;
          s[j][i + n] = see ? __builtin_ldexpf(s[j][i + n] * scale, row_power + c[n]) : kMinusInf;
          sees |= (see ? 1u : 0u) << (16 * j + i + n);
          mx = fmaxf(mx, s[j][i + n]);
        }
      }
    const float less = raise(mx);
    const float f = __builtin_ldexpf(1.0f, 127 + X + kMixedShift - v_ref);
#pragma unroll
    for (int n = 0; n < kWaves; n++) {
      bf16x8 p[NP + 1];
      half8_t seen;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        float e = __builtin_amdgcn_exp2f(s[n >> 1][8 * (n & 1) + i] - less);
        l += e;
        e *= f;
#pragma unroll
        for (int k = 0; k <= NP; k++) {
          p[k][i] = (__bf16)e;
          e -= (float)p[k][i];
        }
        seen[i] = sees >> (8 * n + i) & 1 ? (_Float16)1.0f : (_Float16)0.0f;
      }
#pragma unroll
      for (int t = 0; t < 2 * ND; t++) {
        s16x8 v = value_operand(b, n, t);
        f32x16 count;
        if (nans) {
          half8_t bad;
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const bool is = (v[i] & 0x7FFF) > 0x7F80;
            bad[i] = is ? (_Float16)1.0f : (_Float16)0.0f;
            v[i] = is ? (short)0 : v[i];
          }
#pragma unroll
          for (int i = 0; i < 16; i++) count[i] = 0.0f;
          count = __builtin_amdgcn_mfma_f32_32x32x16_f16(bad, seen, count, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k <= NP; k++)
          acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v), p[k],
                                                           acc[t], 0, 0, 0);
        if (nans) {
#pragma unroll
          for (int i = 0; i < 16; i++)
            if (count[i] > 0.0f) acc[t][i] = __builtin_nanf("");
        }
        __builtin_amdgcn_sched_barrier(0);  // or all operands are read at once
      }
    }
  };

  // a tile again, under references that are right for it or, where a page is none,
  // as a mixed one; seldom more than once
  const auto stage_again = [&](int t, bool absent) __attribute__((always_inline)) {
    load_pages(t);
    load(t);
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < PASSES; p++)
      top = pk_max(top, d.ok[WHOLE ? 0 : p] ? scale_rank(d.ks[p]) | scale_rank(d.vs[p]) << 16 : 0);
    top = wave_pk_max(top);
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    if (!absent) {
      top = pk_max(pk_max(tops[0], tops[1]), pk_max(tops[2], tops[3]));
      top = (uint32_t)__builtin_amdgcn_readfirstlane((int)top);
      k_ref = reference(k_ref, top & 0xFFFF);
      refer(reference(v_ref, top >> 16));
    }
    stage(t, absent);
    __syncthreads();
    load_pages(t + 1);
    load(t + 1);
    load_pages(t + 2);
  };

  if (w.first < w.last) {
    load_pages(w.first);
    load(w.first);
    load_pages(w.first + 1);
    stage(w.first, is_mixed(w.first));
    load(w.first + 1);
    load_pages(w.first + 2);
  }
  __syncthreads();
  for (int t = w.first; t < w.last; t++) {
    const int b = t & 1, first = w.begin + t * kTile;
    bool mixed = is_mixed(t);
    uint32_t any;
    int v_top;
    const auto read = [&]() __attribute__((always_inline)) {
      const u32x4 words = *reinterpret_cast<const u32x4 *>(&staged[b][0]);
      any = (uint32_t)__builtin_amdgcn_readfirstlane((int)(words[0] | words[1] | words[2] | words[3]));
      v_top = __builtin_amdgcn_readfirstlane((int)(max(max(words[0], words[1]), max(words[2], words[3])) >> 8));
    };
    read();
    if (!mixed && (any & (kOver | kNearK | kNearV | kAbsent)) != (kNearK | kNearV)) {
      mixed = (any & kAbsent) != 0;
      stage_again(t, mixed);
      if (mixed) read();
    }
    if (mixed && v_top > v_ref + kMixedReach) refer(v_top - kMixedReach);
    const bool sees = active && max(first, one.lo) <= min(first + kTile - 1, two.hi);
    bool there = true;
    for (int p = 0; p < (WHOLE ? 1 : PASSES); p++) there &= d.ok[p];
    if (sees && !mixed && t + 1 < w.last && !is_mixed(t + 1) && __builtin_amdgcn_ballot_w64(!there) == 0) {
      compute(b, std::true_type{});
      load(t + 2);  // in a branch, it would be waited for where the branches meet
      load_pages(t + 3);
    } else {
      if (t + 1 < w.last) {
        stage(t + 1, is_mixed(t + 1));
        load(t + 2);  // in a branch, it would be waited for where the branches meet
        load_pages(t + 3);
      }
      if (sees) {
        if (mixed) compute_mixed(b, first, (any & kNan) != 0);
        else compute(b, std::false_type{});
      }
    }
    __syncthreads();
  }

  // the row's sums; a lane has dims 8 (i / 4) + 4 half + i % 4 of each 32
  l = add_partner_row<64>(l);
  const int out_row = w.r0 + 32 * wave + r32;
  if (out_row > last_row) return;
  const int head = w.kv_head * a.group + row - token * a.group;
  const bool whole = w.splits == 1;
  const int64_t part = part_row<kRows>(a, w, w.split, 32 * wave + r32);
  if (!whole && half == 0) part_stats(a)[part] = make_float2(m, l);
#pragma unroll
  for (int t = 0; t < 2 * ND; t++)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int c = 32 * t + 2 * i + 4 * half;
      f32x4 v;
#pragma unroll
      for (int n = 0; n < 4; n++) v[n] = __builtin_ldexpf(acc[t][i + n], v_ref - X - 127 - kSumExponent);
      if (32 * t < D) {
        if (whole) store_y4(a, (int64_t)(w.seq.q0 + token) * a.y_stride + (int64_t)head * D + c, quotient(v, l));
        else *reinterpret_cast<f32x4 *>(a.partial + part * D + c) = v;
      }
    }
}

}  // namespace

hipError_t attention_tiled_launch(const AttentionArgs &a, int blocks, hipStream_t stream) {
  const int nd = (a.head_dim + 63) / 64;
#define GO(NP, F, ND)                                                                          \
  if (a.page_size % kWaveKeys == 0)                                                            \
    hipLaunchKernelGGL((attention_tiled_kernel<NP, F, ND, true>), dim3(blocks),                \
                       dim3(kWaves * 64), 0, stream, a);                                       \
  else                                                                                         \
    hipLaunchKernelGGL((attention_tiled_kernel<NP, F, ND, false>), dim3(blocks),               \
                       dim3(kWaves * 64), 0, stream, a)
#define BY_DIM(NP, F)                    \
  switch (nd) {                          \
    case 1: GO(NP, F, 1); break;         \
    case 2: GO(NP, F, 2); break;         \
    case 3: GO(NP, F, 3); break;         \
    default: GO(NP, F, 4); break;        \
  }
  if (a.type == MX_F32) {
    if (a.format == MX_FP4) { BY_DIM(2, MX_FP4) } else { BY_DIM(2, MX_FP8) }
  } else {
    if (a.format == MX_FP4) { BY_DIM(1, MX_FP4) } else { BY_DIM(1, MX_FP8) }
  }
#undef BY_DIM
#undef GO
  return hipGetLastError();
}

}  // namespace q4k
