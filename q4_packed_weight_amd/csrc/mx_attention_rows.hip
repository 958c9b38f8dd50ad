// mx_attention_rows.hip -- attention over a paged MX cache for few rows: the
// (token, head) pairs of one key head's group, 16 at a time.
#include <algorithm>

#include "mx_attention.h"

namespace q4k {
namespace {

constexpr int kWaves = 4;
constexpr int kRows = 16;
constexpr int kStepKeys = 32;

// One wave's 32 keys (lane: key l % 16 of two tiles, group g = l / 16 of its
// dims: 64 p + 16 g .. + 15 for p < ND) as they lie in memory.
template <int FMT, int ND, bool FOURS> struct StepData {
  static constexpr int W = FMT == MX_FP8 ? 4 : 2;  // dwords of 16 codes
  uint32_t k[2][ND][W], v[2][ND][W];
  RawScales<ND, FOURS> ks[2], vs[2];
  uint32_t ok;  // bit by key, the same in every lane
};

// Waves that a SIMD holds at a time: as many as keep a lane's registers (codes,
// queries, sums) from memory.
template <int NP, int ND>
constexpr int kWavesPerSimd = ND == 1 ? 5 : ND == 2 ? (NP == 1 ? 4 : 3) : ND == 3 ? 2 : 1;

// Scores are products S^T = K Q^T of 16 keys by 16 rows: a lane's result is of
// its row l % 16 and keys 4g .. 4g+3, so that a row's statistics are a lane's
// own, and after exp2 the eight weights of two tiles are, as they stand, the
// operand of O^T += V^T P^T with the keys in that order.  V goes through LDS
// as fp16, each wave its own 32 keys, and comes back transposed.  A wave takes
// every fourth step of its workgroup's range; once a step's codes are operands
// and in LDS, the next one's are sent for, and its weights and sums are made
// while they come.  The four results, and those of the shares, are joined by
// their largest x.  Bound by memory and, for small batches, by its latency: 64
// tokens over 1024 .. 8192 keys of 8 heads of 128 (MX_FP8, 621 MB) 140 us, 4.4 TB/s;
// 2 tokens over 131072 keys in MX_FP4 (213 MB) 55 us; one over 1000 keys 10.5 us, of
// which the join is 4: starts, pages and codes are three loads that wait for one
// another, and a step alone on its SIMD takes 1.5 us.
template <int NP, int FMT, int ND, bool MIXED, bool FOURS>
__global__ __launch_bounds__(kWaves * 64, MIXED ? 1 : (kWavesPerSimd<NP, ND>)) void attention_rows_kernel(AttentionArgs a) {
  constexpr int DP = 64 * ND;                // dims, padded
  constexpr int VS = 2 * DP + 32;            // bytes of a key's row of V in LDS
  constexpr int OS = DP + 4;                 // floats of a row of the result
  constexpr int kRegion = kStepKeys * VS > kRows * OS * 4 ? kStepKeys * VS : kRows * OS * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * kRegion];
  __shared__ float2 stats[kWaves][kRows];
  __shared__ __attribute__((aligned(16))) int powers[kWaves][kStepKeys];
  Work w;
  if (!work_of<kRows, kStepKeys>(a, blockIdx.x, w)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const int D = a.head_dim, nb = D / 32;
  const int64_t code_row = FMT == MX_FP8 ? D : D / 2;
  bool has[ND];
#pragma unroll
  for (int p = 0; p < ND; p++) has[p] = 64 * p + 16 * g < D;

  const int32_t *const table = a.table + (int64_t)w.index * a.pages_per_seq;
  // pages of a step's keys; those of keys that no row sees are not used
  const auto load_pages = [&](int step, int (&page)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const int key = w.begin + step * kStepKeys + 16 * j + r16;
      page[j] = table[a.by_page.of(min(max(key, w.any.lo), w.any.hi))];
    }
  };
  int pages[2];
  if (w.first + wave < w.last) load_pages(w.first + wave, pages);

  // queries: rows behind the last one are its copies
  const int row = w.r0 + min(r16, w.rows - 1);
  const int token = a.by_group.of(row);
  const Range mine = w.seq.sees(a, token);
  RawQ<NP> raw[ND][2];
  {
    const int64_t at = (int64_t)(w.seq.q0 + token) * a.q_stride +
                       (int64_t)(w.kv_head * a.group + row - token * a.group) * D;
#pragma unroll
    for (int p = 0; p < ND; p++)
#pragma unroll
      for (int h = 0; h < 2; h++) raw[p][h] = load_q8<NP>(a, at + (has[p] ? 64 * p + 16 * g : 0) + 8 * h);
  }
  // Every lane loads, absent keys and dims row 0 of their head and dims 0 of
  // their row, without a branch; fill_in puts zeros there.
  const bool odd = (D & 32) != 0;
  StepData<FMT, ND, FOURS> d;
  const auto load_step = [&](int step, const int (&page)[2]) __attribute__((always_inline)) {
    uint32_t okay = 0;
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const int key = w.begin + step * kStepKeys + 16 * j + r16;
      const bool ok = step < w.last && key >= w.any.lo && key <= w.any.hi &&
                      (uint32_t)page[j] < (uint32_t)a.n_pages;
      okay |= ((uint32_t)__builtin_amdgcn_ballot_w64(ok) & 0xFFFFu) << (16 * j);
      const uint32_t place = key - a.by_page.of(key) * a.page_size;
      const uint32_t r = ok ? (page[j] * a.n_kv_heads + w.kv_head) * a.page_size + place : 0;
      const uint64_t at = (uint64_t)r * code_row, s_at = (uint64_t)r * nb;
#pragma unroll
      for (int p = 0; p < ND; p++) {
        const int c = (has[p] ? 64 * p + 16 * g : 0) * (FMT == MX_FP8 ? 2 : 1) / 2;
        load_codes(a.k_codes + at + c, d.k[j][p]);
        load_codes(a.v_codes + at + c, d.v[j][p]);
      }
      d.ks[j].load(a.k_scales + s_at, nb, g);
      d.vs[j].load(a.v_scales + s_at, nb, g);
    }
    d.ok = (uint32_t)__builtin_amdgcn_readfirstlane((int)okay);
  };
  const auto fill_in = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; j++) {
      d.ks[j].settle(g);
      d.vs[j].settle(g);
    }
    if (d.ok != 0xFFFFFFFFu || odd) {
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const bool ok = d.ok >> (16 * j + r16) & 1;
#pragma unroll
        for (int p = 0; p < ND; p++) {
          if (!ok || !has[p]) {
#pragma unroll
            for (int i = 0; i < StepData<FMT, ND, FOURS>::W; i++) d.k[j][p][i] = d.v[j][p][i] = 0;
            d.ks[j].clear(p);
            d.vs[j].clear(p);
          }
        }
      }
    }
  };

  if (w.first + wave < w.last) {
    load_step(w.first + wave, pages);
    load_pages(w.first + wave + kWaves, pages);
  }
  half8_t q[NP][ND][2];
  int row_power;
  {
    float f[ND][2][8];
    uint32_t amax = 0;
#pragma unroll
    for (int p = 0; p < ND; p++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        q8_to_f32<NP>(a, raw[p][h], f[p][h]);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          if (!has[p]) f[p][h][i] = 0.0f;
          const uint32_t b = __builtin_bit_cast(uint32_t, f[p][h][i]) & 0x7FFFFFFFu;
          amax = b > amax ? b : amax;
        }
      }
    amax = swap_max_u32(amax);
    const int e = row_exponent(amax);
    row_power = e + a.scale_power;
#pragma unroll
    for (int p = 0; p < ND; p++)
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float v = amax >= 0x7F800000u ? __builtin_nanf("") : __builtin_ldexpf(f[p][h][i], -e);
          q[0][p][h][i] = (_Float16)v;
          if constexpr (NP == 2) q[1][p][h][i] = (_Float16)(v - (float)q[0][p][h][i]);
        }
  }

  f32x4 acc[4 * ND];
#pragma unroll
  for (int i = 0; i < 4 * ND; i++) acc[i] = f32x4{0, 0, 0, 0};
  float m = kMinusInf, l = 0.0f;
  bool any_held = false;  // then stats has rows' m without and what is held back
  int v_ref = kFirstRef;
  uint8_t *const mem = lds + wave * kRegion;
  typedef __attribute__((address_space(3))) s16x4 LdsS16x4;
  const uint8_t *const read_at = mem + (4 * g + (r16 >> 2)) * VS + 8 * (r16 & 3);
  constexpr int X = kCodeExponent<FMT>;
  constexpr int W = StepData<FMT, ND, FOURS>::W;

  // 16 dims of 32 values, transposed
  const auto value_operand = [&](int t) __attribute__((always_inline)) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4 *)(read_at + 32 * t));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4 *)(read_at + 32 * t + 16 * VS));
    return s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  // scores of the step's keys, their blocks scaled by f
  const auto scores = [&](const float (&f)[2][ND], f32x4 (&s)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; j++) {
      s[j] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int p = 0; p < ND; p++) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const half8_t k = codes_operand<FMT>(&d.k[j][p][h * W / 2], f[j][p]);
#pragma unroll
          for (int n = 0; n < NP; n++)
            s[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[n][p][h], s[j], 0, 0, 0);
        }
      }
    }
  };
  // The values of x go into the maximum, and what was summed is scaled to the new
  // one and to the new reference; a maximum that is up to 2^4 too low stays, as
  // the weights' 2^14 still are fp16.
  const auto raise = [&](const float (&x)[8], int v_new) __attribute__((always_inline)) {
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < 8; i++) mx = fmaxf(mx, x[i]);
    mx = swap_max32(swap_max16(mx));
    if (__builtin_amdgcn_ballot_w64(mx - m > kMostExponent) != 0 || v_new != v_ref) {
      int power = v_ref - v_new;
      if (power > 0 || (power < 0 && any_held)) {
        float2 kept = make_float2(m, 0.0f);
        if (any_held) kept = stats[wave][r16];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 16 * ND; i++) top = max(top, sum_bits(acc[i >> 2][i & 3]));
        power += (int)kept.y;
        const int more = held_back(swap_max_u32(top), power);
        power -= more;
        l = __builtin_ldexpf(l, (int)kept.y - more);
        m = kept.x + more;
        any_held = __builtin_amdgcn_ballot_w64(more != 0) != 0;
        if (any_held) stats[wave][r16] = make_float2(kept.x, more);
      }
      v_ref = v_new;
      const bool up = mx - m > kMostExponent;
      const float to = up ? exponent_base(mx) : m, f = up ? __builtin_amdgcn_exp2f(m - to) : 1.0f;
      l *= f;
#pragma unroll
      for (int i = 0; i < 16 * ND; i++)
        acc[i >> 2][i & 3] = __builtin_ldexpf(acc[i >> 2][i & 3] * f, power);
      m = to;
      if (any_held && up) stats[wave][r16] = make_float2(m, 0.0f);
    }
    return m == kMinusInf ? 0.0f : m;
  };

  // Keys that all rows see (or none: absent ones).  The references stay as long
  // as no scale of the step is above them and one at least is no more than 2^8
  // below, which each lane compares for itself; else they are made anew.
  int k_ref = kFirstRef;
  const auto compute = [&](int step) __attribute__((always_inline)) {
    uint32_t k_top = 0, v_top = 0;
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int p = 0; p < d.ks[j].S; p++) {
        k_top = pk_max(k_top, d.ks[j].pair[p]);
        v_top = pk_max(v_top, d.vs[j].pair[p]);
      }
    k_top = max(k_top & 0xFFFF, k_top >> 16);
    v_top = max(v_top & 0xFFFF, v_top >> 16);
    int v_new = v_ref;
    bool nans = false;
    if (__builtin_amdgcn_ballot_w64((int)k_top > k_ref || (int)v_top > v_ref) != 0 ||
        (k_ref != kLastRef && __builtin_amdgcn_ballot_w64((int)k_top + 8 >= k_ref) == 0) ||
        (v_ref != kLastRef && __builtin_amdgcn_ballot_w64((int)v_top + 8 >= v_ref) == 0)) {
      nans = __builtin_amdgcn_ballot_w64(max(k_top, v_top) == 255) != 0;
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 2; j++)
#pragma unroll
        for (int p = 0; p < ND; p++)
          top = pk_max(top, scale_rank(d.ks[j].of(p)) | scale_rank(d.vs[j].of(p)) << 16);
      top = wave_pk_max(top);
      k_ref = reference(k_ref, (int)(top & 0xFFFF));
      v_new = reference(v_ref, (int)(top >> 16));
    }
    float kf[2][ND], vf[2][ND];
#pragma unroll
    for (int j = 0; j < 2; j++) {
      d.ks[j].powers(127 + X - k_ref, kf[j]);
      d.vs[j].powers(127 + X - v_new, vf[j]);
    }
    if (nans) {
#pragma unroll
      for (int j = 0; j < 2; j++)
#pragma unroll
        for (int p = 0; p < ND; p++) {
          if (d.ks[j].of(p) == 255) kf[j][p] = __builtin_nanf("");
          if (d.vs[j].of(p) == 255) vf[j][p] = __builtin_nanf("");
        }
    }
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int p = 0; p < ND; p++) {
        uint8_t *const to = mem + (16 * j + r16) * VS + (64 * p + 16 * g) * 2;
        *reinterpret_cast<half8_t *>(to) = codes_operand<FMT>(&d.v[j][p][0], vf[j][p]);
        *reinterpret_cast<half8_t *>(to + 16) = codes_operand<FMT>(&d.v[j][p][W / 2], vf[j][p]);
      }
    __builtin_amdgcn_wave_barrier();
    f32x4 s[2];
    scores(kf, s);
    const uint32_t ok = d.ok;
    load_step(step + kWaves, pages);
    load_pages(step + 2 * kWaves, pages);
    const float c = score_scale(a.scale, row_power + k_ref - X - 127);
    float x[8];
    {  // rounded as its maximum is: no product with x - m
#pragma clang fp contract(off)
#pragma unroll
      for (int i = 0; i < 8; i++) x[i] = s[i >> 2][i & 3] * c;
    }
    if (ok != 0xFFFFFFFFu) {
#pragma unroll
      for (int i = 0; i < 8; i++)
        x[i] = ok >> (16 * (i >> 2) + 4 * g + (i & 3)) & 1 ? x[i] : kMinusInf;
    }
    const float less = raise(x, v_new);
    half8_t p[NP];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float e = __builtin_amdgcn_exp2f(x[i] - less);
      l += e;
      p[0][i] = (_Float16)e;
      if constexpr (NP == 2) p[1][i] = (_Float16)(e - (float)p[0][i]);
    }
#pragma unroll
    for (int t = 0; t < 4 * ND; t++) {
      const half8_t v = __builtin_bit_cast(half8_t, value_operand(t));
#pragma unroll
      for (int n = 0; n < NP; n++)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p[n], acc[t], 0, 0, 0);
    }
    __builtin_amdgcn_wave_barrier();
  };

  // keys that some rows see and others do not: no reference may come from a key
  // that a row does not see, and no NaN
  const auto compute_mixed = [&](int step) __attribute__((always_inline)) {
    uint32_t rank[2], v_top = 0;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < 2; j++) {
      rank[j] = 0;
#pragma unroll
      for (int p = 0; p < ND; p++) {
        rank[j] = max(rank[j], scale_rank(d.ks[j].of(p)));
        v_top = max(v_top, scale_rank(d.vs[j].of(p)));
        nan |= has_nan<FMT>(d.v[j][p], d.vs[j].of(p));
        const float s = block_scale(d.vs[j].of(p), -kMixedShift);
        uint8_t *const to = mem + (16 * j + r16) * VS + (64 * p + 16 * g) * 2;
        *reinterpret_cast<bf16x8 *>(to) = codes_operand_bf16<FMT>(&d.v[j][p][0], s);
        *reinterpret_cast<bf16x8 *>(to + 16) = codes_operand_bf16<FMT>(&d.v[j][p][W / 2], s);
      }
      rank[j] = swap_max_u32(rank[j]);
      if (g == 0) powers[wave][16 * j + r16] = (int)rank[j] - X - 127;
    }
    __builtin_amdgcn_wave_barrier();
    float kf[2][ND];
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int p = 0; p < ND; p++) kf[j][p] = block_scale(d.ks[j].of(p), 127 + X - (int)rank[j]);
    f32x4 s[2];
    scores(kf, s);
    const uint32_t ok = d.ok;
    load_step(step + kWaves, pages);
    load_pages(step + 2 * kWaves, pages);
    const int first = w.begin + step * kStepKeys;
    float x[8];
    half8_t sees;
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const i32x4 c = *reinterpret_cast<const i32x4 *>(&powers[wave][16 * j + 4 * g]);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int n = 16 * j + 4 * g + i, key = first + n;
        const bool see = (ok >> n & 1) != 0 && key >= mine.lo && key <= mine.hi;
        x[4 * j + i] = see ? __builtin_ldexpf(s[j][i] * a.scale, row_power + c[i]) : kMinusInf;
        sees[4 * j + i] = see ? (_Float16)1.0f : (_Float16)0.0f;
      }
    }
    int v_new = v_ref;
    if (__builtin_amdgcn_ballot_w64((int)v_top > v_ref + kMixedReach) != 0)
      v_new = (int)wave_pk_max(v_top) - kMixedReach;
    const float less = raise(x, v_new);
    const float power = __builtin_ldexpf(1.0f, 127 + X + kMixedShift - v_ref);
    // as many bf16 as hold what fp16 holds of them in the other form
    bf16x8 p[NP + 1];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      float e = __builtin_amdgcn_exp2f(x[i] - less);
      l += e;
      e *= power;
#pragma unroll
      for (int n = 0; n <= NP; n++) {
        p[n][i] = (__bf16)e;
        e -= (float)p[n][i];
      }
    }
    const bool nans = __builtin_amdgcn_ballot_w64(nan) != 0;
#pragma unroll
    for (int t = 0; t < 4 * ND; t++) {
      s16x8 v = value_operand(t);
      f32x4 count = {0, 0, 0, 0};
      if (nans) {
        // 0 * NaN is NaN: the NaNs taken out, and a row's dims in which it sees
        // one counted by a product of zeros and ones
        half8_t bad;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const bool is = (v[i] & 0x7FFF) > 0x7F80;
          bad[i] = is ? (_Float16)1.0f : (_Float16)0.0f;
          v[i] = is ? (short)0 : v[i];
        }
        count = __builtin_amdgcn_mfma_f32_16x16x32_f16(bad, sees, count, 0, 0, 0);
      }
#pragma unroll
      for (int n = 0; n <= NP; n++)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v), p[n], acc[t],
                                                         0, 0, 0);
      if (nans) {
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (count[i] > 0.0f) acc[t][i] = __builtin_nanf("");
      }
    }
    __builtin_amdgcn_wave_barrier();
  };
  for (int step = w.first + wave; step < w.last; step += kWaves) {
    fill_in();
    const int one = w.begin + step * kStepKeys;
    if (MIXED && (max(one, w.any.lo) < w.all.lo || min(one + kStepKeys - 1, w.any.hi) > w.all.hi))
      compute_mixed(step);
    else
      compute(step);
  }

  // the waves' results, under one power
  l = add_partner_row<64>(add_partner_row<32>(l));
  float *const o = reinterpret_cast<float *>(mem) + r16 * OS;
#pragma unroll
  for (int t = 0; t < 4 * ND; t++) {
    f32x4 v = acc[t];
#pragma unroll
    for (int i = 0; i < 4; i++)
      v[i] = __builtin_ldexpf(v[i], v_ref - kCodeExponent<FMT> - 127 - kSumExponent);
    *reinterpret_cast<f32x4 *>(o + 16 * t + 4 * g) = v;
  }
  if (g == 0) stats[wave][r16] = make_float2(m, l);
  __syncthreads();
  const int out = threadIdx.x >> 4;  // row
  if (out >= w.rows) return;
  float most = kMinusInf, sum = 0.0f, share[kWaves];
#pragma unroll
  for (int i = 0; i < kWaves; i++) most = fmaxf(most, stats[i][out].x);
#pragma unroll
  for (int i = 0; i < kWaves; i++) {
    share[i] = part_share(stats[i][out].x, most);
    sum += share[i] * stats[i][out].y;
  }
  const int out_row = w.r0 + out, out_token = a.by_group.of(out_row);
  const int head = w.kv_head * a.group + out_row - out_token * a.group;
  const bool whole = w.splits == 1;
  const int64_t part = part_row<kRows>(a, w, w.split, out);
  if (!whole && (threadIdx.x & 15) == 0) part_stats(a)[part] = make_float2(most, sum);
  for (int c = 4 * (threadIdx.x & 15); c < D; c += 64) {
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kWaves; i++)
      v += share[i] * *reinterpret_cast<const f32x4 *>(lds + i * kRegion + (out * OS + c) * 4);
    if (whole) {
      store_y4(a, (int64_t)(w.seq.q0 + out_token) * a.y_stride + (int64_t)head * D + c,
               quotient(v, sum));
    } else {
      *reinterpret_cast<f32x4 *>(a.partial + part * D + c) = v;
    }
  }
}

// Rows of a workgroup of the join: one a wave of the few, four of the many, whose
// workgroups take longer to start than to work (mixed batch of 52 tiles and 5 heads
// 13 us, with two rows 20).
constexpr int join_rows(int rows) { return rows == kRows ? 4 : 16; }

// The shares' results joined, a wave to a row: the weights of 64 shares at a
// time, then four dims of every second share to a lane (of all for head_dim
// above 128, of every fourth up to 64).
template <int ROWS, int KEYS>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a) {
  constexpr int kChunk = join_rows(ROWS), kWide = ROWS == kRows ? 8 : 2;  // many rows: few shares
  Work w;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, D = a.head_dim;
  if (!work_of<ROWS, KEYS, true>(a, blockIdx.x, w) || w.splits == 1 ||
      w.unit + w.splits > a.units)  // starts that are not ascending
    return;
  const int width = D > 128 ? 64 : D > 64 ? 32 : 16, groups = 64 / width;
  const int c = lane & (width - 1), g = lane / width, columns = D / 4;
  const int64_t stride = (int64_t)a.n_kv_heads * ROWS;
  for (int r = kChunk * blockIdx.y + wave; r < min(w.rows, kChunk * ((int)blockIdx.y + 1)); r += 4) {
    const int row = w.r0 + r, token = a.by_group.of(row);
    const int head = w.kv_head * a.group + row - token * a.group;
    const int64_t part = part_row<ROWS>(a, w, 0, r);
    const float2 *const stats = part_stats(a) + part;
    const f32x4 *const values = reinterpret_cast<const f32x4 *>(a.partial + part * D) + min(c, columns - 1);
    float m = kMinusInf, total = 0.0f;
    f32x4 v = {0, 0, 0, 0};
    for (int from = 0; from < w.splits; from += 64) {
      const int n = min(64, w.splits - from);
      const float2 mine = lane < n ? stats[(from + lane) * stride] : make_float2(kMinusInf, 0.0f);
      float most = mine.x;
#pragma unroll
      for (int i = 1; i < 64; i *= 2) most = fmaxf(most, __shfl_xor(most, i));
      most = fmaxf(most, m);
      const float share = lane < n ? part_share(mine.x, most) : 0.0f, before = part_share(m, most);
      total = total * before + group_sum<64>(share * mine.y);
      v *= before;
      // kWide parts on their way at a time; those behind the last are the last, times 0
      for (int i = g; i - g < n; i += kWide * groups) {
        f32x4 part[kWide];
#pragma unroll
        for (int k = 0; k < kWide; k++)
          part[k] = values[(from + min(i + k * groups, n - 1)) * stride * columns];
#pragma unroll
        for (int k = 0; k < kWide; k++) {
          const int at = i + k * groups;
          const float f = __shfl(share, at & 63);
          v += (at < n ? f : 0.0f) * part[k];
        }
      }
      m = most;
    }
    for (int i = width; i < 64; i *= 2) {
#pragma unroll
      for (int k = 0; k < 4; k++) v[k] += __shfl_xor(v[k], i);
    }
    if (g == 0 && c < columns)
      store_y4(a, (int64_t)(w.seq.q0 + token) * a.y_stride + (int64_t)head * D + 4 * c,
               quotient(v, total));
  }
}

// More than one tile of 16 rows: the form for many rows.  64 tokens over 4096 keys of
// 4 heads of 128 (MX_FP8, 280 MB): 70 us with 8 rows a head, 154 with 32 here, of
// which three quarters of a 128-row tile are idle.
bool tiled(const AttentionArgs &a) { return (int64_t)a.max_queries * a.group > kRows; }

// Workgroups on the chip at a time.
int slots(const AttentionArgs &a) {
  const int nd = (a.head_dim + 63) / 64;
  if (tiled(a)) return 256 * (nd <= 2 ? 2 : 1);
  return 256 * (nd <= 2 ? 4 : 2);
}
template <int NP, int FMT, int ND>
void launch_rows(const AttentionArgs &a, int blocks, hipStream_t stream) {
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(blocks), dim3(256), 0, stream, a); };
  if constexpr (ND % 2 == 0) {
    if (a.head_dim % 128 == 0) {
      if (a.max_queries == 1) go(attention_rows_kernel<NP, FMT, ND, false, true>);
      else go(attention_rows_kernel<NP, FMT, ND, true, true>);
      return;
    }
  }
  if (a.max_queries == 1) go(attention_rows_kernel<NP, FMT, ND, false, false>);
  else go(attention_rows_kernel<NP, FMT, ND, true, false>);
}
constexpr int kMaxPlanned = 512;  // sequences that every workgroup looks through

}  // namespace

// Tiles are laid out by the sequences' own sizes where those are few enough to
// look through; keys are cut into shares where the tiles alone are fewer than
// twice (many rows: once) the workgroups that run at a time.  With more tiles, or
// more sequences, each tile's keys are one workgroup's: of 256 tokens with 8 heads, one
// over 131072 keys and the others over 500, that one takes 1.2 ms (of 200, cut, all
// take 0.11); 500 and 600 over 500 to 600 keys each take 117 and 133 us, 5.2 TB/s.
int64_t mx_attention_workspace_bytes(AttentionArgs &a) {
  const int rows = tiled(a) ? kTiledRows : kRows, keys = tiled(a) ? kTiledKeys : kStepKeys;
  a.tiles = (int)(((int64_t)a.max_queries * a.group + rows - 1) / rows);
  a.by_tiles = FastDiv(a.tiles);
  a.by_kv_heads = FastDiv(a.n_kv_heads);
  a.planned = a.n_seqs <= kMaxPlanned;
  a.shares_wanted = 0;
  a.n_parts = 0;
  int64_t tiles = (int64_t)a.n_seqs * a.tiles;
  if (a.planned) tiles = std::min(tiles, (int64_t)a.n_tokens * a.group / rows + a.n_seqs);
  a.units = (int)tiles;
  const int64_t steps = ((int64_t)a.pages_per_seq * a.page_size + keys - 1) / keys;
  const int64_t limit = slots(a) * (tiled(a) ? 1 : 2);
  if (!a.planned || tiles * a.n_kv_heads >= limit || steps * keys <= kMinKeys ||
      steps * tiles > 0x7FFFFFFF)
    return 0;
  // a sequence's last share is shorter than the others: half a share each
  const int64_t want = std::max(tiles, (slots(a) - tiles * a.n_kv_heads / 2) / a.n_kv_heads);
  const int64_t most = tiles * (steps * keys / kMinKeys + 1);  // units if all are of kMinKeys
  a.shares_wanted = (int)want;
  a.units = (int)std::min(tiles + want, most);
  a.n_parts = (int64_t)a.units * a.n_kv_heads * rows;
  return (a.n_parts * (a.head_dim + 2) * 4 + 255) / 256 * 256;
}

hipError_t mx_attention_launch(const AttentionArgs &a, hipStream_t stream) {
  const int blocks = a.units * a.n_kv_heads;
  hipError_t e;
  if (tiled(a)) {
    e = attention_tiled_launch(a, blocks, stream);
  } else {
    const int nd = (a.head_dim + 63) / 64;
#define GO(NP, F, ND)                                                                           \
  launch_rows<NP, F, ND>(a, blocks, stream)
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
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.n_parts == 0) return e;
  const int64_t rows = (int64_t)a.max_queries * a.group;
  const int64_t tiles = std::min((int64_t)a.n_seqs * a.tiles,
                                 (int64_t)a.n_tokens * a.group / (tiled(a) ? kTiledRows : kRows) + a.n_seqs);
  const int chunk = join_rows(tiled(a) ? kTiledRows : kRows);
  const dim3 grid((uint32_t)(tiles * a.n_kv_heads),
                  (uint32_t)((std::min<int64_t>(rows, tiled(a) ? kTiledRows : kRows) + chunk - 1) / chunk));
  if (tiled(a))
    hipLaunchKernelGGL((attention_join_kernel<kTiledRows, kTiledKeys>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((attention_join_kernel<kRows, kStepKeys>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace q4k
