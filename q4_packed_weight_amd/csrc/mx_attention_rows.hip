// mx_attention_rows.hip -- attention over a paged MX cache for few rows: the
// (token, head) pairs of one key head's group, 16 at a time.
#include "mx_attention.h"

namespace q4k {
namespace {

constexpr int kWaves = 4;
constexpr int kRows = 16;
constexpr int kStepKeys = 32;

// One wave's 32 keys (lane: key l % 16 of two tiles, group g = l / 16 of its
// dims: 64 p + 16 g .. + 15 for p < ND) as they lie in memory.
template <int FMT, int ND> struct StepData {
  static constexpr int W = FMT == MX_FP8 ? 4 : 2;  // dwords of 16 codes
  uint32_t k[2][ND][W], v[2][ND][W];
  uint32_t ks[2][ND], vs[2][ND];
  uint32_t ok;  // bit by key, the same in every lane
};

// Scores are products S^T = K Q^T of 16 keys by 16 rows: a lane's result is of
// its row l % 16 and keys 4g .. 4g+3, so that a row's statistics are a lane's
// own, and after exp2 the eight weights of two tiles are, as they stand, the
// operand of O^T += V^T P^T with the keys in that order.  V goes through LDS
// as fp16, each wave its own 32 keys, and comes back transposed.  A wave takes
// every fourth step of its workgroup's range, the next one's codes in flight;
// the four results, and those of the ranges, are joined by their largest x.
template <int NP, int FMT, int ND>
__global__ __launch_bounds__(kWaves * 64) void attention_rows_kernel(AttentionArgs a) {
  constexpr int DP = 64 * ND;                // dims, padded
  constexpr int VS = 2 * DP + 32;            // bytes of a key's row of V in LDS
  constexpr int OS = DP + 4;                 // floats of a row of the result
  constexpr int kRegion = kStepKeys * VS > kRows * OS * 4 ? kStepKeys * VS : kRows * OS * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * kRegion];
  __shared__ float2 stats[kWaves][kRows];
  __shared__ __attribute__((aligned(16))) float powers[kWaves][kStepKeys];
  Work w;
  if (!work_of<kRows, kStepKeys>(a, blockIdx.x, a.splits, w) || w.split >= w.splits) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const int D = a.head_dim, nb = D / 32;
  const int64_t code_row = FMT == MX_FP8 ? D : D / 2;
  bool has[ND];
#pragma unroll
  for (int p = 0; p < ND; p++) has[p] = 64 * p + 16 * g < D;

  // queries: rows behind the last one are its copies
  const int row = w.r0 + min(r16, w.rows - 1);
  const int token = a.by_group.of(row);
  const Range mine = w.seq.sees(a, token);
  half8_t q[NP][ND][2];
  float row_scale;
  {
    const int64_t at = (int64_t)(w.seq.q0 + token) * a.q_stride +
                       (int64_t)(w.kv_head * a.group + row - token * a.group) * D;
    float f[ND][2][8];
    uint32_t amax = 0;
#pragma unroll
    for (int p = 0; p < ND; p++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        if (has[p]) load_q8(a, at + 64 * p + 16 * g + 8 * h, f[p][h]);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          if (!has[p]) f[p][h][i] = 0.0f;
          const uint32_t b = __builtin_bit_cast(uint32_t, f[p][h][i]) & 0x7FFFFFFFu;
          amax = b > amax ? b : amax;
        }
      }
    amax = swap_max_u32(amax);
    const int e = row_exponent(amax);
    row_scale = amax >= 0x7F800000u ? __builtin_nanf("") : __builtin_ldexpf(a.scale, e);
#pragma unroll
    for (int p = 0; p < ND; p++)
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float v = __builtin_ldexpf(f[p][h][i], -e);
          q[0][p][h][i] = (_Float16)v;
          if constexpr (NP == 2) q[1][p][h][i] = (_Float16)(v - (float)q[0][p][h][i]);
        }
  }

  const int32_t *const table = a.table + (int64_t)w.index * a.pages_per_seq;
  const auto load_step = [&](int step, StepData<FMT, ND> &d) {
    uint32_t okay = 0;
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const int key = w.begin + step * kStepKeys + 16 * j + r16;
      bool ok = step < w.last && key >= w.any.lo && key <= w.any.hi;
      int page = 0, at = 0;
      if (ok) {
        at = a.by_page.of(key);
        page = table[at];
        ok = page >= 0 && page < a.n_pages;
      }
      const int64_t r = ((int64_t)page * a.n_kv_heads + w.kv_head) * a.page_size +
                        (key - at * a.page_size);
      okay |= ((uint32_t)__builtin_amdgcn_ballot_w64(ok) & 0xFFFFu) << (16 * j);
#pragma unroll
      for (int p = 0; p < ND; p++) {
        d.ks[j][p] = d.vs[j][p] = 0;
#pragma unroll
        for (int i = 0; i < StepData<FMT, ND>::W; i++) d.k[j][p][i] = d.v[j][p][i] = 0;
        if (ok && has[p]) {
          const int64_t c = r * code_row + (64 * p + 16 * g) * (FMT == MX_FP8 ? 2 : 1) / 2;
          const int64_t s = r * nb + 2 * p + (g >> 1);
          load_codes(a.k_codes + c, d.k[j][p]);
          load_codes(a.v_codes + c, d.v[j][p]);
          d.ks[j][p] = a.k_scales[s];
          d.vs[j][p] = a.v_scales[s];
        }
      }
    }
    d.ok = (uint32_t)__builtin_amdgcn_readfirstlane((int)okay);
  };

  f32x4 acc[4 * ND];
#pragma unroll
  for (int i = 0; i < 4 * ND; i++) acc[i] = f32x4{0, 0, 0, 0};
  float m = kMinusInf, l = 0.0f;
  int v_ref = kFirstValueRef;
  uint8_t *const mem = lds + wave * kRegion;
  typedef __attribute__((address_space(3))) s16x4 LdsS16x4;
  const uint8_t *const read_at = mem + (4 * g + (r16 >> 2)) * VS + 8 * (r16 & 3);
  constexpr int X = kCodeExponent<FMT>;
  constexpr int W = StepData<FMT, ND>::W;

  // 16 dims of 32 values, transposed
  const auto value_operand = [&](int t) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4 *)(read_at + 32 * t));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4 *)(read_at + 32 * t + 16 * VS));
    return s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  // scores of the step's keys under the scales that `base(j)` gives tile j
  const auto scores = [&](const StepData<FMT, ND> &d, const auto &base, f32x4 (&s)[2]) {
#pragma unroll
    for (int j = 0; j < 2; j++) {
      s[j] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int p = 0; p < ND; p++) {
        const float f = block_scale(d.ks[j][p], base(j));
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const half8_t k = codes_operand<FMT>(&d.k[j][p][h * W / 2], f);
#pragma unroll
          for (int n = 0; n < NP; n++)
            s[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[n][p][h], s[j], 0, 0, 0);
        }
      }
    }
  };
  // the values of x go into the maximum; what was summed is scaled to the new one
  // and to the new reference
  const auto raise = [&](const float (&x)[8], int v_new) {
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < 8; i++) mx = fmaxf(mx, x[i]);
    mx = swap_max32(swap_max16(mx));
    const float m_new = fmaxf(m, mx);
    if (__builtin_amdgcn_ballot_w64(m_new > m) != 0 || v_new != v_ref) {
      const float f = m_new > m ? __builtin_amdgcn_exp2f(m - m_new) : 1.0f;
      l *= f;
      const float o = __builtin_ldexpf(f, v_ref - v_new);
#pragma unroll
      for (int i = 0; i < 4 * ND; i++) acc[i] *= o;
      m = m_new;
      v_ref = v_new;
    }
    return (m == kMinusInf ? 0.0f : m) - kWeightExponent;
  };

  // keys that all rows see (or none: absent ones)
  const auto compute = [&](const StepData<FMT, ND> &d) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int p = 0; p < ND; p++)
        top = pk_max(top, scale_rank(d.ks[j][p]) | scale_rank(d.vs[j][p]) << 16);
    top = wave_pk_max(top);
    const int k_ref = top & 0xFFFF, v_new = value_ref(v_ref, (int)(top >> 16));
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int p = 0; p < ND; p++) {
        const float s = block_scale(d.vs[j][p], 127 + X - v_new);
        uint8_t *const to = mem + (16 * j + r16) * VS + (64 * p + 16 * g) * 2;
        *reinterpret_cast<half8_t *>(to) = codes_operand<FMT>(&d.v[j][p][0], s);
        *reinterpret_cast<half8_t *>(to + 16) = codes_operand<FMT>(&d.v[j][p][W / 2], s);
      }
    __builtin_amdgcn_wave_barrier();
    f32x4 s[2];
    scores(d, [&](int) { return 127 + X - k_ref; }, s);
    const float c = __builtin_ldexpf(row_scale, k_ref - X - 127);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = s[i >> 2][i & 3] * c;
    if (d.ok != 0xFFFFFFFFu) {
#pragma unroll
      for (int i = 0; i < 8; i++)
        x[i] = d.ok >> (16 * (i >> 2) + 4 * g + (i & 3)) & 1 ? x[i] : kMinusInf;
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
  const auto compute_mixed = [&](int step, const StepData<FMT, ND> &d) {
    uint32_t rank[2];
    bool nan = false;
#pragma unroll
    for (int j = 0; j < 2; j++) {
      rank[j] = 0;
#pragma unroll
      for (int p = 0; p < ND; p++) {
        rank[j] = max(rank[j], scale_rank(d.ks[j][p]));
        nan |= has_nan<FMT>(d.v[j][p], d.vs[j][p]);
        const float s = block_scale(d.vs[j][p], 127 + X - v_ref);
        uint8_t *const to = mem + (16 * j + r16) * VS + (64 * p + 16 * g) * 2;
        *reinterpret_cast<bf16x8 *>(to) = codes_operand_bf16<FMT>(&d.v[j][p][0], s);
        *reinterpret_cast<bf16x8 *>(to + 16) = codes_operand_bf16<FMT>(&d.v[j][p][W / 2], s);
      }
      rank[j] = swap_max_u32(rank[j]);
      if (g == 0) powers[wave][16 * j + r16] = __builtin_ldexpf(1.0f, (int)rank[j] - X - 127);
    }
    __builtin_amdgcn_wave_barrier();
    f32x4 s[2];
    scores(d, [&](int j) { return 127 + X - (int)rank[j]; }, s);
    const int first = w.begin + step * kStepKeys;
    float x[8];
    half8_t sees;
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const f32x4 c = *reinterpret_cast<const f32x4 *>(&powers[wave][16 * j + 4 * g]);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int n = 16 * j + 4 * g + i, key = first + n;
        const bool see = (d.ok >> n & 1) != 0 && key >= mine.lo && key <= mine.hi;
        x[4 * j + i] = see ? s[j][i] * row_scale * c[i] : kMinusInf;
        sees[4 * j + i] = see ? (_Float16)1.0f : (_Float16)0.0f;
      }
    }
    const float less = raise(x, v_ref);
    // as many bf16 as hold what fp16 holds of them in the other form
    bf16x8 p[NP + 1];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      float e = __builtin_amdgcn_exp2f(x[i] - less);
      l += e;
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
  const auto take = [&](int step, const StepData<FMT, ND> &d) {
    const int one = w.begin + step * kStepKeys;
    if (max(one, w.any.lo) < w.all.lo || min(one + kStepKeys - 1, w.any.hi) > w.all.hi)
      compute_mixed(step, d);
    else
      compute(d);
  };

  StepData<FMT, ND> d0, d1;
  int step = w.first + wave;
  load_step(step, d0);
  while (step < w.last) {
    load_step(step + kWaves, d1);
    take(step, d0);
    step += kWaves;
    if (step >= w.last) break;
    load_step(step + kWaves, d0);
    take(step, d1);
    step += kWaves;
  }

  // the waves' results, each as it stands before its power is put back
  l = add_partner_row<64>(add_partner_row<32>(l));
  float *const o = reinterpret_cast<float *>(mem) + r16 * OS;
#pragma unroll
  for (int t = 0; t < 4 * ND; t++) {
    f32x4 v = acc[t];
#pragma unroll
    for (int i = 0; i < 4; i++)
      v[i] = __builtin_ldexpf(v[i], v_ref - kCodeExponent<FMT> - 127);
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
  const int64_t flat = (int64_t)(w.seq.q0 + out_token) * a.n_kv_heads * a.group + head;
  const bool whole = w.splits == 1;
  if (!whole && (threadIdx.x & 15) == 0)
    reinterpret_cast<float2 *>(a.partial + a.n_rows * a.splits * D)[flat * a.splits + w.split] =
        make_float2(most, sum);
  for (int c = 4 * (threadIdx.x & 15); c < D; c += 64) {
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kWaves; i++)
      v += share[i] * *reinterpret_cast<const f32x4 *>(lds + i * kRegion + (out * OS + c) * 4);
    if (whole) {
      v *= sum == 0.0f ? 0.0f : 1.0f / sum;
      store_y4(a, (int64_t)(w.seq.q0 + out_token) * a.y_stride + (int64_t)head * D + c, v);
    } else {
      *reinterpret_cast<f32x4 *>(a.partial + (flat * a.splits + w.split) * D + c) = v;
    }
  }
}

// The ranges' results joined, a row to 16 lanes.
template <int ROWS, int KEYS>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a) {
  Work w;
  if (!work_of<ROWS, KEYS>(a, blockIdx.x, 1, w) || w.splits == 1) return;
  const int out = 16 * blockIdx.y + (threadIdx.x >> 4), D = a.head_dim;
  if (out >= w.rows) return;
  const int row = w.r0 + out, token = a.by_group.of(row);
  const int head = w.kv_head * a.group + row - token * a.group;
  const int64_t flat = (int64_t)(w.seq.q0 + token) * a.n_kv_heads * a.group + head;
  const float2 *const stats =
      reinterpret_cast<const float2 *>(a.partial + a.n_rows * a.splits * D) + flat * a.splits;
  float most = kMinusInf, sum = 0.0f;
  for (int i = 0; i < w.splits; i++) most = fmaxf(most, stats[i].x);
  for (int i = 0; i < w.splits; i++) sum += part_share(stats[i].x, most) * stats[i].y;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  for (int c = 4 * (threadIdx.x & 15); c < D; c += 64) {
    f32x4 v = {0, 0, 0, 0};
    for (int i = 0; i < w.splits; i++)
      v += part_share(stats[i].x, most) *
           *reinterpret_cast<const f32x4 *>(a.partial + (flat * a.splits + i) * D + c);
    store_y4(a, (int64_t)(w.seq.q0 + token) * a.y_stride + (int64_t)head * D + c, v * inv);
  }
}

// More than one tile of 16 rows: the form for many rows.
bool tiled(const AttentionArgs &a) { return (int64_t)a.max_queries * a.group > kRows; }

}  // namespace

// Ranges of keys so that about four workgroups come to a CU, none for fewer
// than kMinKeys keys.
int64_t mx_attention_workspace_bytes(AttentionArgs &a) {
  const int rows = tiled(a) ? kTiledRows : kRows;
  a.tiles = (int)(((int64_t)a.max_queries * a.group + rows - 1) / rows);
  const int64_t blocks = (int64_t)a.n_seqs * a.tiles * a.n_kv_heads;
  const int64_t most = (int64_t)a.pages_per_seq * a.page_size / kMinKeys;
  const int64_t want = (tiled(a) ? 512 : 1024) / blocks;
  a.splits = (int)(want < most ? (want > 1 ? want : 1) : (most > 1 ? most : 1));
  a.by_tiles = FastDiv(a.tiles);
  a.by_splits = FastDiv(a.splits);
  return a.splits == 1 ? 0 : (a.n_rows * a.splits * (a.head_dim + 2) * 4 + 255) / 256 * 256;
}

hipError_t mx_attention_launch(const AttentionArgs &a, hipStream_t stream) {
  const int blocks = a.n_seqs * a.tiles * a.n_kv_heads;
  hipError_t e;
  if (tiled(a)) {
    e = attention_tiled_launch(a, blocks * a.splits, stream);
  } else {
    const int nd = (a.head_dim + 63) / 64;
#define GO(NP, F, ND)                                                                         \
  hipLaunchKernelGGL((attention_rows_kernel<NP, F, ND>), dim3(blocks * a.splits), dim3(256), 0, \
                     stream, a)
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
  if (e != hipSuccess || a.splits == 1) return e;
  if (tiled(a))
    hipLaunchKernelGGL((attention_join_kernel<kTiledRows, kTiledKeys>), dim3(blocks, kTiledRows / 16),
                       dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((attention_join_kernel<kRows, kStepKeys>), dim3(blocks), dim3(256), 0, stream,
                       a);
  return hipGetLastError();
}

}  // namespace q4k
