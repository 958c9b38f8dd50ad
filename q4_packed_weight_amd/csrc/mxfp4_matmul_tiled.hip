// mxfp4_matmul_tiled.hip -- the MX product for many tokens: tiles staged
// through LDS for the scaled matrix instruction.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mx_internal.h"
#include "mx_lds.h"

namespace q4k {
namespace {

// BM tokens x BN weight rows per workgroup of WM x WN waves, each with
// TM x TN tiles of 16x16; S stages of KS 128-position steps in LDS, loaded by
// DMA (no registers, every wave's loads in flight across the barriers).
// Weights are the A operand as they lie, tokens the B operand, both with their
// scale bytes: nothing is decoded.  ALIGNED: rows of whole steps whose scales
// start at dwords.
// 256x256 tiles are bound by the matrix pipe and the loads from beyond the L2
// taking turns imperfectly (8192^3: loads alone 255 us, products alone 300,
// together 367, 3.0 PFLOP/s; 4096 tokens, 14336 x 4096: 182 us, 2.64 PFLOP/s,
// where four rounds of tiles do not fill 256 CUs evenly; fp32 outputs, two
// instructions a product, 347 us); 64x64 ones by
// the latency of their few stages (64 tokens, 14336 x 4096: 13.0 us).
template <int AF, int T, int WM, int WN, int TM, int TN, int KS, int S, bool ALIGNED>
__global__ __launch_bounds__(64 * WM * WN, 2) void mxfp4_tiled_kernel(
    const uint8_t *a, const uint8_t *as, const uint8_t *w, const uint8_t *ws, void *y, int M,
    int64_t K, int64_t N, int tiles_m, int tiles_n) {
  constexpr int kW = WM * WN, kThreads = 64 * kW;
  constexpr bool kHalves = kW == 8;
  constexpr int BM = 16 * WM * TM, BN = 16 * WN * TN;
  constexpr int AP = kTileLoads<AF>;
  constexpr int kStepLoads = BM / 16 * AP + BN / 16;      // 1 KiB each
  constexpr int kMine = kStepLoads / kW;                  // of a wave, tokens first
  constexpr int kMineA = BM / 16 * AP / kW;
  constexpr int kStep = kStepLoads * 1024;
  // Scales are kept for kChunk steps at a time, 4 kChunk bytes a row.
  constexpr int kChunk = KS == 2 ? 8 : 4;
  constexpr int kScales = (BM + BN) * 4 * kChunk;
  constexpr int kScaleLoads = kScales / 1024 / kW;        // of a wave
  static_assert(BM / 16 * AP % kW == 0 && BN / 16 % kW == 0 && BM % 64 == 0 && BN % 64 == 0,
                "whole loads");
  static_assert(!kHalves || (KS == 1 && S == 3 && BM + BN <= kThreads), "");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S * KS * kStep + 2 * kScales];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;

  // Workgroups go to the 8 XCDs in turn: each XCD takes a run of tiles, eight
  // token tiles deep, so that its L2 serves the tiles that share operands.
  const int tiles = tiles_m * tiles_n;
  int id = blockIdx.x;
  {
    const int per = tiles / 8, more = tiles % 8, x = id & 7;
    id = (id >> 3) + x * per + (x < more ? x : more);
  }
  constexpr int kDeep = 8;
  const int group = id / (kDeep * tiles_n), in = id % (kDeep * tiles_n);
  const int deep = tiles_m - group * kDeep < kDeep ? tiles_m - group * kDeep : kDeep;
  const int bm = group * kDeep + in % deep, bn = in / deep;
  const int m0 = bm * BM;
  const int64_t n0 = (int64_t)bn * BN;
  const int rows_m = M - m0 < BM ? M - m0 : BM, rows_n = N - n0 < BN ? (int)(N - n0) : BN;

  const int nb = (int)(K / 32);
  const int steps = (nb + 3) / 4;
  const uint32_t a_bytes = (uint32_t)(AF == MX_FP4 ? K / 2 : K), w_bytes = (uint32_t)(K / 2);
  const i32x4 a_view = buffer_view(a + (int64_t)m0 * a_bytes, rows_m * a_bytes);
  const i32x4 w_view = buffer_view(w + n0 * w_bytes, rows_n * w_bytes);
  const auto token = [&](int m) { return m < rows_m ? m : rows_m - 1; };
  const auto weight_row = [&](int n) { return n < rows_n ? n : rows_n - 1; };

  uint32_t offset[kMine];
#pragma unroll
  for (int i = 0; i < kMine; i++) {
    const int p = i * kW + wave;
    if (i < kMineA)
      offset[i] = (uint32_t)token(p * (16 / AP) + tile_row<AF>(lane)) * a_bytes +
                  16 * tile_chunk<AF>(lane);
    else
      offset[i] = (uint32_t)weight_row(paired_row(p - BM / 16 * AP, tile_row<MX_FP4>(lane))) *
                      w_bytes + 16 * tile_chunk<MX_FP4>(lane);
  }
  const uint32_t lds0 = lds_address(lds);
  // The loads of stage u: its KS steps, zeros past the row's end.
  const auto issue = [&](int u, int buf) {
#pragma unroll
    for (int k = 0; k < KS; k++) {
      const int s = u * KS + k;
#pragma unroll
      for (int i = 0; i < kMine; i++) {
        const int p = i * kW + wave;
        const bool is_a = i < kMineA;
        uint32_t o = offset[i] + (uint32_t)s * (is_a ? 64 * AP : 64);
        if (KS > 1 || 4 * s + 4 > nb) {
          const int block = is_a ? chunk_block<AF>(tile_chunk<AF>(lane)) : tile_chunk<MX_FP4>(lane);
          if (4 * s + block >= nb) o = kPastEnd;
        }
        load16_to_lds(is_a ? a_view : w_view, o, lds0 + (buf * KS + k) * kStep + p * 1024);
      }
    }
  };

  // Scales: `row` counts the tile's tokens, then its weight rows.
  uint8_t *const scales = lds + S * KS * kStep;
  const auto scale_row = [&](int row) {
    return row < BM ? as + (int64_t)(m0 + token(row)) * nb
                    : ws + (n0 + weight_row(row - BM)) * nb;
  };
  // From step s on, through registers into one of the two halves: 16 bytes of
  // a row a thread, at any alignment.
  constexpr int kParts = kChunk / 4;                      // of a row
  constexpr int kHold = (BM + BN) * kParts / kThreads > 0 ? (BM + BN) * kParts / kThreads : 1;
  u32x4 held[kHold];
  const auto load_scales = [&](int s) {
#pragma unroll
    for (int i = 0; i < kHold; i++) {
      const int part = tid + i * kThreads;
      if (part < (BM + BN) * kParts)
        held[i] = load_scales16(scale_row(part / kParts), 4 * (int64_t)s + part % kParts * 16, nb);
    }
  };
  const auto store_scales = [&](int half) {
#pragma unroll
    for (int i = 0; i < kHold; i++) {
      const int part = tid + i * kThreads;
      if (part < (BM + BN) * kParts)
        *reinterpret_cast<u32x4 *>(scales + half * kScales + part * 16) =
            kHalves ? transpose_bytes(held[i]) : held[i];
    }
  };
  // The same straight into LDS, for rows whose scales start at dwords.
  const i32x4 as_view = buffer_view(as + (int64_t)m0 * nb, rows_m * nb);
  const i32x4 ws_view = buffer_view(ws + n0 * nb, rows_n * nb);
  const auto issue_scales = [&](int s, int half) {
    constexpr int kRows = 64 / kParts;                    // of a load
#pragma unroll
    for (int i = 0; i < kScaleLoads; i++) {
      const int p = i * kW + wave;
      const bool is_a = p < BM / kRows;
      const int row = p * kRows + lane / kParts;
      const uint32_t o = (uint32_t)(is_a ? token(row) : weight_row(row - BM)) * nb + 4 * s +
                         lane % kParts * 16;
      load16_to_lds(is_a ? as_view : ws_view, o,
                    lds0 + S * KS * kStep + half * kScales + p * 1024);
    }
  };

  const int wm = wave % WM, wn = wave / WM;
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; i++)
#pragma unroll
    for (int j = 0; j < TN; j++) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int sa[TM], sw[TN];
  typedef Operand<AF> Tokens[TM];
  typedef Operand<MX_FP4> Weights[TN];
  const auto fetch = [&](const uint8_t *st, Tokens &ta, Weights &tw) {
#pragma unroll
    for (int i = 0; i < TM; i++)
      ta[i] = read_operand<AF>(st + (wm * TM + i) * AP * 1024, operand_at<AF>(r, g));
#pragma unroll
    for (int j = 0; j < TN; j++)
      tw[j] = read_operand<MX_FP4>(st + (BM / 16 * AP + wn * TN + j) * 1024,
                                   operand_at<MX_FP4>(r, g));
  };
  // The scales of steps s .. s+3 (a multiple of four), one to a byte; kHalves,
  // which has no registers for four dwords a tile, keeps them so.  A stage of
  // two steps multiplies both where the row has only the first: the second's
  // codes are zeros, and its scales are held at 1, as the bytes behind a row's
  // are the next row's, whose 255 would make these zeros NaN.
  const auto fetch_scales = [&](int s) {
    const uint8_t *sc = scales + (s / kChunk % 2) * kScales + s % kChunk * 4;
    const uint32_t which = byte_of_two(g);
    const uint32_t past = KS == 1 || s + 4 <= steps ? 0u : ~0u << (8 * (steps - s));
    const auto one = [&](int row) {
      const uint8_t *p = sc + row * 4 * kChunk;
      if constexpr (kHalves) return *reinterpret_cast<const int *>(p + 4 * g);
      const uint32_t v = byte_of_four(*reinterpret_cast<const u32x4 *>(p), which);
      return (int)((v & ~past) | (0x7F7F7F7Fu & past));
    };
#pragma unroll
    for (int i = 0; i < TM; i++) sa[i] = one((wm * TM + i) * 16 + r);
#pragma unroll
    for (int j = 0; j < TN; j++) sw[j] = one(BM + paired_row(wn * TN + j, r));
  };
  const auto multiply = [&](const Tokens &ta, const Weights &tw, auto jc) {
    constexpr int J = decltype(jc)::value;
    if constexpr (T == MX_F32 && AF == MX_FP8) {  // tokens outside: each is split in two once
#pragma unroll
      for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++)
          acc[i][j] = mfma_mx<MX_FP4, AF, true, J>(eight(tw[j]), eight(ta[i]), acc[i][j], sw[j],
                                                   sa[i]);
    } else {
#pragma unroll
      for (int j = 0; j < TN; j++)
#pragma unroll
        for (int i = 0; i < TM; i++)
          acc[i][j] = mfma_mx<MX_FP4, AF, false, J>(eight(tw[j]), eight(ta[i]), acc[i][j], sw[j],
                                                    sa[i]);
    }
  };

  const int stages = (steps + KS - 1) / KS;
  if (!ALIGNED || kHalves) {
    load_scales(0);
    store_scales(0);
  } else {
    issue_scales(0, 0);
  }
#pragma unroll
  for (int u = 0; u < S - 1; u++)
    if (u < stages) issue(u, u);
  int buf = 0;
  if constexpr (kHalves) {
    // Each SIMD holds one wave of the first four and one of the others, and
    // the second four run one barrier behind: while one wave of a SIMD
    // multiplies a step, the other fetches its operands from LDS and sends
    // the loads of two steps on.  A stage is overwritten after both halves
    // have fetched from it, and read after the barrier that follows every
    // wave's wait for it.
    if (steps > 1) wait_loads<kMine>();
    else wait_loads<0>();
    lds_barrier();
    const bool behind = wave >= 4;
    if (behind) lds_barrier();
    const auto step = [&](int s, auto jc) {
      constexpr int J = decltype(jc)::value;
      if (J == 3 && s + 1 < steps) store_scales(((s >> 2) + 1) & 1);  // read two barriers on
      Tokens ta;
      Weights tw;
      fetch(lds + buf * kStep, ta, tw);
      if constexpr (J == 0) {
        fetch_scales(s);
        if (s + 4 < steps) load_scales(s + 4);
      }
      if (s + 2 < steps) {
        issue(s + 2, buf == 0 ? 2 : buf - 1);
        wait_loads<kMine>();
      } else {
        wait_loads<0>();
      }
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
      multiply(ta, tw, jc);
      __builtin_amdgcn_sched_barrier(0);
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
      buf = buf == 2 ? 0 : buf + 1;
    };
    for (int s = 0; s < steps; s += 4) {
      step(s, std::integral_constant<int, 0>{});
      if (s + 1 < steps) step(s + 1, std::integral_constant<int, 1>{});
      if (s + 2 < steps) step(s + 2, std::integral_constant<int, 2>{});
      if (s + 3 < steps) step(s + 3, std::integral_constant<int, 3>{});
    }
    if (!behind) lds_barrier();
  } else {
    // Four steps a turn, in 4 / KS stages.  The next chunk of scales is sent
    // for at a chunk's first stage, before the loads of a stage that is waited
    // for within the chunk.
    static_assert(S - 1 <= kChunk / KS && 4 % KS == 0, "");
    const auto stage = [&](int u, auto jc) {
      constexpr int J = decltype(jc)::value;
      const int s = u * KS;
      const bool chunk = J == 0 && s % kChunk == 0 && s + kChunk < steps;
      if (u + S - 2 < stages) wait_loads<(S - 2) * kMine * KS>();
      else wait_loads<0>();
      lds_barrier();
      if (chunk) {
        if constexpr (ALIGNED) issue_scales(s + kChunk, (s / kChunk + 1) % 2);
        else load_scales(s + kChunk);
      }
      if (u + S - 1 < stages) issue(u + S - 1, buf == 0 ? S - 1 : buf - 1);
      if constexpr (J == 0) fetch_scales(s);
      Tokens ta[KS];
      Weights tw[KS];
#pragma unroll
      for (int k = 0; k < KS; k++) fetch(lds + (buf * KS + k) * kStep, ta[k], tw[k]);
      multiply(ta[0], tw[0], jc);
      if constexpr (KS == 2) multiply(ta[1], tw[1], std::integral_constant<int, J + 1>{});
      if (!ALIGNED && chunk) store_scales((s / kChunk + 1) % 2);
      buf = buf == S - 1 ? 0 : buf + 1;
    };
    for (int u = 0; u < stages; u += 4 / KS) {
      stage(u, std::integral_constant<int, 0>{});
      if constexpr (KS == 2) {
        if (u + 1 < stages) stage(u + 1, std::integral_constant<int, 2>{});
      } else {
        if (u + 1 < stages) stage(u + 1, std::integral_constant<int, 1>{});
        if (u + 2 < stages) stage(u + 2, std::integral_constant<int, 2>{});
        if (u + 3 < stages) stage(u + 3, std::integral_constant<int, 3>{});
      }
    }
  }

  const bool wide = N % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
  const auto pair = [&](int i, int j, float (&f)[8]) {
#pragma unroll
    for (int q = 0; q < 4; q++) {
      f[q] = acc[i][j][q];
      f[4 + q] = acc[i][j + 1][q];
    }
  };
  const bool whole = TN >= 4 && wide && rows_m == BM && rows_n == BN;
  if (whole || !wide) {
    // Out through LDS, 16 tokens at a time in a part of the wave's own, so that
    // a store covers whole runs of a token's row: straight from registers it
    // covers pieces of 16 rows.  Whole tiles: 4096x128x16384, 134 MB of bf16
    // outputs, 64 us, so 48, and past the caches 43, as the kernel's end does
    // not wait for their lines to be written back; smaller outputs go the same
    // way, which is not timed apart.  Rows that do not start at
    // 16 bytes go out value by value, 64 neighbours to a store
    // (4096x4096x4097 bf16 110 us, so 85; 333x1056x4097 10.0, so 8.7; 16 bytes
    // at a time between the rows' ends: 95, 10.3).
    typedef typename MxStore<T>::type Out;
    constexpr int kSize = sizeof(Out), kRow = 16 * TN * kSize, kStride = kRow + 16;
    constexpr int kLanes = kRow / 16, kTokens = 64 / kLanes;  // of a store of 16 bytes a lane
    static_assert(kW * 16 * kStride <= (int)sizeof(lds), "");
    const int columns = rows_n - wn * 16 * TN;                // may pass the tile's, or be none
    uint8_t *const part = lds + wave * (16 * kStride);
    lds_barrier();  // every wave's operands are read
#pragma unroll
    for (int i = 0; i < TM; i++) {
      const int first = (wm * TM + i) * 16;
      const auto out_row = [&](int t) {
        return static_cast<Out *>(y) + (int64_t)(m0 + first + t) * N + n0 + wn * 16 * TN;
      };
#pragma unroll
      for (int j = 0; j < TN; j += 2) {
        float f[8];
        pair(i, j, f);
        store_raw8<T>(part + r * kStride + (16 * j + 8 * g) * kSize, 0, f32_to_raw8<T>(f));
      }
      wait_lds();
      if (TN >= 4 && wide) {
#pragma unroll
        for (int q = 0; q < 16 / kTokens; q++) {
          const int t = q * kTokens + lane / kLanes, at = lane % kLanes * 16;
          const u32x4 v = *reinterpret_cast<const u32x4 *>(part + t * kStride + at);
          __builtin_nontemporal_store(
              v, reinterpret_cast<u32x4 *>(reinterpret_cast<uint8_t *>(out_row(t)) + at));
        }
      } else {
#pragma unroll
        for (int c = 0; c < 16 * 16 * TN; c += 64) {
          const int t = (c + lane) / (16 * TN), at = (c + lane) % (16 * TN);
          const Out v = *reinterpret_cast<const Out *>(part + t * kStride + at * kSize);
          if (first + t < rows_m && at < columns) out_row(t)[at] = v;
        }
      }
      wait_lds();  // the part is read
    }
    return;
  }
  // Partial tiles, and tiles whose rows are no longer than what four lanes
  // write, of rows that start at 16 bytes.
#pragma unroll
  for (int i = 0; i < TM; i++) {
    const int m = (wm * TM + i) * 16 + r;
    if (m >= rows_m) continue;
#pragma unroll
    for (int j = 0; j < TN; j += 2) {
      const int n = (wn * TN + j) * 16 + 8 * g;
      float f[8];
      pair(i, j, f);
      store_row8<T>(y, (int64_t)(m0 + m) * N + n0 + n, f, rows_n - n, true);
    }
  }
}

template <int AF, int T, int WM, int WN, int TM, int TN, int KS, int S, bool ALIGNED>
void launch(const uint8_t *a, const uint8_t *as, const uint8_t *w, const uint8_t *ws, int M,
            int64_t K, int64_t N, void *Y, hipStream_t stream) {
  const int tm = (M + 16 * WM * TM - 1) / (16 * WM * TM);
  const int tn = (int)((N + 16 * WN * TN - 1) / (16 * WN * TN));
  hipLaunchKernelGGL((mxfp4_tiled_kernel<AF, T, WM, WN, TM, TN, KS, S, ALIGNED>), dim3(tm * tn),
                     dim3(64 * WM * WN), 0, stream, a, as, w, ws, Y, M, K, N, tm, tn);
}

// The tile by estimated time.  Measured at input_dim 4096, e4m3 tokens, bf16
// outputs (graph replays, us): 64x64 tiles 11.5 up to 256 of them, 18.2 for
// 512, 31 for 1024, 56.6 for 2048; 128x128 tiles 23.4 for 128, 25.0 for 256,
// 39.3 for 512, 68 for 896; 256x256 tiles 44.6 for 64, 48.7 for 224, 186 for
// 896, a whole round of 256 at a time.  Other lengths and formats, and fp32
// outputs, whose products take twice as long, are taken to scale all three
// alike; that is not measured.
template <int AF, int T>
void choose(const uint8_t *a, const uint8_t *as, const uint8_t *w, const uint8_t *ws, int M,
            int64_t K, int64_t N, void *Y, hipStream_t stream) {
  const auto tiles = [&](int b) { return (double)((M + b - 1) / b) * (double)((N + b - 1) / b); };
  const double small = std::max(11.0, 5.0 + 0.0255 * tiles(64));
  const double middle = std::max(23.0, 7.0 + 0.068 * tiles(128));
  const double large = 50.0 * std::ceil(tiles(256) / 256.0);
  const bool aligned = mx_aligned_scales(as, ws, K);
  if (large <= middle && large <= small) {
    launch<AF, T, 4, 2, 4, 8, 1, 3, true>(a, as, w, ws, M, K, N, Y, stream);
  } else if (middle <= small) {
    if (aligned) launch<AF, T, 2, 2, 4, 4, 1, 3, true>(a, as, w, ws, M, K, N, Y, stream);
    else launch<AF, T, 2, 2, 4, 4, 1, 3, false>(a, as, w, ws, M, K, N, Y, stream);
  } else {
    if (aligned) launch<AF, T, 2, 2, 2, 2, 2, 3, true>(a, as, w, ws, M, K, N, Y, stream);
    else launch<AF, T, 2, 2, 2, 2, 2, 3, false>(a, as, w, ws, M, K, N, Y, stream);
  }
}

}  // namespace

hipError_t mxfp4_matmul_tiled_launch(const uint8_t *a, const uint8_t *as, int a_format,
                                     const uint8_t *w, const uint8_t *ws, int64_t M, int64_t K,
                                     int64_t N, void *Y, int type, hipStream_t stream) {
#define CALL(AF)                                                                         \
  switch (type) {                                                                        \
    case MX_F32: choose<AF, MX_F32>(a, as, w, ws, (int)M, K, N, Y, stream); break;       \
    case MX_BF16: choose<AF, MX_BF16>(a, as, w, ws, (int)M, K, N, Y, stream); break;     \
    default: choose<AF, MX_F16>(a, as, w, ws, (int)M, K, N, Y, stream); break;           \
  }
  if (a_format == MX_FP4) { CALL(MX_FP4) } else { CALL(MX_FP8) }
#undef CALL
  return hipGetLastError();
}

}  // namespace q4k
