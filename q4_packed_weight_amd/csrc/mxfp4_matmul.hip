// mxfp4_matmul.hip -- products of MX activations with MXFP4 weights on the
// scaled matrix instructions.
#include <type_traits>

#include "mx_internal.h"
#include "mx_lds.h"

namespace q4k {
namespace {

// 16 NR weight rows x 16 NT tokens per workgroup, for few tokens: each of its
// W waves takes a run of the 128-position steps of input_dim for the whole
// tile, through a ring of S stages of its own in LDS (no barrier until the
// end), and the waves' partial tiles are added in LDS in wave order.  Weights
// are the A operand of the scaled instruction, tokens the B operand; nothing
// is decoded.  Splitting input_dim inside the workgroup rather than over more
// of them needs no second pass, and its loads need no registers.  Bound by the
// weights' bytes and the latency of the first loads (one token, 4096 x 4096,
// 8.9 MB of weights: 4.6 us, of which a launch and the first load are most; 16
// tokens, 14336 x 4096, 31 MB: 10.4 us, 3.0 TB/s).
// ALIGNED: rows of whole steps whose scales start at dwords; they come through
// LDS too, four steps at a time.  Otherwise they come through registers, whose
// wait also waits for the loads in flight.  Rows and tokens past the end read
// the last one and are not stored; positions past the end read as zeros.
// The launch bound is 8 waves' also where W is 4: with a bound of 4 the compiler
// keeps the accumulators in AGPRs and copies them around every product that
// holds its operands (14336 x 8192, 64 tokens, fp32: 37.5 us, now 31.6).
template <int AF, int T, int NR, int NT, int W, int S, bool ALIGNED>
__global__ __launch_bounds__(512) void mxfp4_rows_kernel(
    const uint8_t *a, const uint8_t *as, const uint8_t *w, const uint8_t *ws, void *y, int M,
    int64_t K, int64_t N) {
  constexpr int AP = kTileLoads<AF>;
  constexpr int kLoads = NT * AP + NR;                            // of a step
  constexpr int kRing = (S * kLoads + (ALIGNED ? 2 : 0)) * 1024;  // and of four steps' scales
  constexpr int kSum = NR * NT * 1024;
  constexpr int kWave = kRing > kSum ? kRing : kSum;              // a wave's part of LDS
  static_assert(NR <= 2 && NT <= 4 && S >= 2 && S <= 4, "");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[W * kWave];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int nb = (int)(K / 32);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NR);
  const int m0 = blockIdx.y * (16 * NT);
  const int rows_n = N - n0 < 16 * NR ? (int)(N - n0) : 16 * NR;
  const int rows_m = M - m0 < 16 * NT ? M - m0 : 16 * NT;
  const uint32_t a_bytes = (uint32_t)(AF == MX_FP4 ? K / 2 : K), w_bytes = (uint32_t)(K / 2);
  const i32x4 a_view = buffer_view(a + (int64_t)m0 * a_bytes, rows_m * a_bytes);
  const i32x4 w_view = buffer_view(w + n0 * w_bytes, rows_n * w_bytes);
  const i32x4 as_view = buffer_view(as + (int64_t)m0 * nb, rows_m * nb);
  const i32x4 ws_view = buffer_view(ws + n0 * nb, rows_n * nb);
  const auto token = [&](int m) { return m < rows_m ? m : rows_m - 1; };
  const auto weight_row = [&](int tile, int row) {
    const int n = NR % 2 == 0 ? paired_row(tile, row) : 16 * tile + row;
    return n < rows_n ? n : rows_n - 1;
  };

  const int steps = (nb + 3) / 4;
  const int first = (int)((int64_t)steps * wave / W);
  const int last = (int)((int64_t)steps * (wave + 1) / W);
  uint8_t *const mine = lds + wave * kWave;
  uint8_t *const scales = mine + S * kLoads * 1024;
  const uint32_t ring = lds_address(mine);

  uint32_t a_at[NT * AP], w_at[NR];
#pragma unroll
  for (int i = 0; i < NT * AP; i++)
    a_at[i] = (uint32_t)token(i * (16 / AP) + tile_row<AF>(lane)) * a_bytes +
              16 * tile_chunk<AF>(lane);
#pragma unroll
  for (int i = 0; i < NR; i++)
    w_at[i] = (uint32_t)weight_row(i, tile_row<MX_FP4>(lane)) * w_bytes +
              16 * tile_chunk<MX_FP4>(lane);
  const auto issue = [&](int s, int buf) {
    const uint32_t to = ring + buf * (kLoads * 1024);
    const bool in_a = ALIGNED || 4 * s + chunk_block<AF>(tile_chunk<AF>(lane)) < nb;
    const bool in_w = ALIGNED || 4 * s + tile_chunk<MX_FP4>(lane) < nb;
#pragma unroll
    for (int i = 0; i < NR; i++)
      load16_to_lds(w_view, in_w ? w_at[i] + 64u * s : kPastEnd, to + (NT * AP + i) * 1024);
#pragma unroll
    for (int i = 0; i < NT * AP; i++)
      load16_to_lds(a_view, in_a ? a_at[i] + 64u * AP * s : kPastEnd, to + i * 1024);
  };
  // 16 scale bytes (four steps) of row r of tile g: one load for the tokens'
  // tiles, one for the weights'
  const uint32_t as_at = g < NT ? (uint32_t)token(16 * g + r) * nb : kPastEnd;
  const uint32_t ws_at = g < NR ? (uint32_t)weight_row(g, r) * nb : kPastEnd;
  const auto issue_scales = [&](int s) {
    load16_to_lds(as_view, g < NT ? as_at + 4 * s : kPastEnd, ring + S * kLoads * 1024);
    load16_to_lds(ws_view, g < NR ? ws_at + 4 * s : kPastEnd, ring + (S * kLoads + 1) * 1024);
  };

  f32x4 acc[NR][NT];
#pragma unroll
  for (int i = 0; i < NR; i++)
#pragma unroll
    for (int t = 0; t < NT; t++) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (first < last) {
    int buf = 0, sa[NT], sw[NR];
    u32x4 next_a[NT], next_w[NR];
    const auto load_scales = [&](int s) {
#pragma unroll
      for (int t = 0; t < NT; t++)
        next_a[t] = load_scales16(as + (int64_t)(m0 + token(16 * t + r)) * nb, 4 * (int64_t)s, nb);
#pragma unroll
      for (int i = 0; i < NR; i++)
        next_w[i] = load_scales16(ws + (n0 + weight_row(i, r)) * nb, 4 * (int64_t)s, nb);
    };
    if constexpr (ALIGNED) issue_scales(first);
    else load_scales(first);
#pragma unroll
    for (int d = 0; d < S - 1; d++)
      if (first + d < last) issue(first + d, d);
    const auto step = [&](int s, auto jc) {
      constexpr int J = decltype(jc)::value;
      wait_lds();  // the stage and the scales that the next loads overwrite are read
      if constexpr (ALIGNED && J == 1) {
        if (s + 3 < last) issue_scales(s + 3);
      }
      if (s + S - 1 < last) issue(s + S - 1, buf == 0 ? S - 1 : buf - 1);
      // The scales of the steps from s on are older than stage s.
      const int ahead = last - 1 - s;
      if (S > 3 && ahead >= 3) wait_loads<(S > 3 ? 3 : 0) * kLoads>();
      else if (S > 2 && ahead >= 2) wait_loads<(S > 2 ? 2 : 0) * kLoads>();
      else if (ahead >= 1) wait_loads<kLoads>();
      else wait_loads<0>();
      if constexpr (J == 0) {
        const uint32_t which = byte_of_two(g);
#pragma unroll
        for (int t = 0; t < NT; t++) {
          if constexpr (ALIGNED)
            next_a[t] = *reinterpret_cast<const u32x4 *>(scales + t * 256 + r * 16);
          sa[t] = (int)byte_of_four(next_a[t], which);
        }
#pragma unroll
        for (int i = 0; i < NR; i++) {
          if constexpr (ALIGNED)
            next_w[i] = *reinterpret_cast<const u32x4 *>(scales + 1024 + i * 256 + r * 16);
          sw[i] = (int)byte_of_four(next_w[i], which);
        }
        if (!ALIGNED && s + 4 < last) load_scales(s + 4);
      }
      const uint8_t *st = mine + buf * (kLoads * 1024);
      Operand<MX_FP4> wv[NR];
#pragma unroll
      for (int i = 0; i < NR; i++)
        wv[i] = read_operand<MX_FP4>(st + (NT * AP + i) * 1024, operand_at<MX_FP4>(r, g));
#pragma unroll
      for (int t = 0; t < NT; t++) {
        const Operand<AF> v = read_operand<AF>(st + t * AP * 1024, operand_at<AF>(r, g));
#pragma unroll
        for (int i = 0; i < NR; i++)
          acc[i][t] = mfma_mx<MX_FP4, AF, T == MX_F32, J>(eight(wv[i]), eight(v), acc[i][t], sw[i], sa[t]);
      }
      buf = buf == S - 1 ? 0 : buf + 1;
    };
    for (int s = first; s < last; s += 4) {
      step(s, std::integral_constant<int, 0>{});
      if (s + 1 < last) step(s + 1, std::integral_constant<int, 1>{});
      if (s + 2 < last) step(s + 2, std::integral_constant<int, 2>{});
      if (s + 3 < last) step(s + 3, std::integral_constant<int, 3>{});
    }
    wait_lds();
  }
#pragma unroll
  for (int i = 0; i < NR; i++)
#pragma unroll
    for (int t = 0; t < NT; t++)
      *reinterpret_cast<f32x4 *>(mine + (i * NT + t) * 1024 + lane * 16) = acc[i][t];
  __syncthreads();

  const auto sum = [&](int tile) {
    const uint8_t *p = lds + tile * 1024 + lane * 16;
    f32x4 d = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
    for (int i = 1; i < W; i++) d += *reinterpret_cast<const f32x4 *>(p + i * kWave);
    return d;
  };
  if constexpr (NR % 2 == 0) {
    const bool wide = N % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
    for (int q = wave; q < NR / 2 * NT; q += W) {
      const int i = q / NT * 2, t = q % NT;
      const f32x4 lo = sum(i * NT + t), hi = sum((i + 1) * NT + t);
      const float f[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      const int m = 16 * t + r, n = 16 * i + 8 * g;
      if (m < rows_m) store_row8<T>(y, (int64_t)(m0 + m) * N + n0 + n, f, rows_n - n, wide);
    }
  } else {
    for (int q = wave; q < NR * NT; q += W) {
      const f32x4 d = sum(q);
      const int m = 16 * (q % NT) + r, n = 16 * (q / NT) + 4 * g;
      if (m >= rows_m) continue;
#pragma unroll
      for (int k = 0; k < 4; k++)
        if (n + k < rows_n) store_value<T>(y, (int64_t)(m0 + m) * N + n0 + n + k, d[k]);
    }
  }
}

template <int AF, int T>
void launch_rows(const uint8_t *a, const uint8_t *as, const uint8_t *w, const uint8_t *ws, int M,
                 int64_t K, int64_t N, void *Y, hipStream_t stream) {
  const bool aligned = mx_aligned_scales(as, ws, K);
  const auto run = [&](auto nr, auto nt, auto nw, auto ns) {
    constexpr int NR = decltype(nr)::value, NT = decltype(nt)::value;
    constexpr int W = decltype(nw)::value, S = decltype(ns)::value;
    const dim3 grid((unsigned)((N + 16 * NR - 1) / (16 * NR)), (M + 16 * NT - 1) / (16 * NT));
    if (aligned)
      hipLaunchKernelGGL((mxfp4_rows_kernel<AF, T, NR, NT, W, S, true>), grid, dim3(W * 64), 0,
                         stream, a, as, w, ws, Y, M, K, N);
    else
      hipLaunchKernelGGL((mxfp4_rows_kernel<AF, T, NR, NT, W, S, false>), grid, dim3(W * 64), 0,
                         stream, a, as, w, ws, Y, M, K, N);
  };
  typedef std::integral_constant<int, 1> I1;
  typedef std::integral_constant<int, 2> I2;
  typedef std::integral_constant<int, 3> I3;
  typedef std::integral_constant<int, 4> I4;
  typedef std::integral_constant<int, 8> I8;
  // About as many workgroups as CUs; wider tiles read the tokens less often.
  // At input_dim 4096 (graph replays): 1x4096 4.4 us, 16x14336 10.5,
  // 32x4096 6.0, 24x8192 6.9, 64x4096 8.1, 64x8192 9.4.
  if (M <= 16) {
    if (N <= 4096) run(I1{}, I1{}, I8{}, I4{});
    else run(I2{}, I1{}, I4{}, I4{});
  } else if (M <= 32) {
    if (N <= 4096) run(I1{}, I2{}, I8{}, I3{});
    else run(I2{}, I2{}, I4{}, I3{});
  } else {
    if (N <= 4096) run(I1{}, I4{}, I8{}, I2{});
    else run(I2{}, I4{}, I4{}, I3{});
  }
}

}  // namespace

hipError_t mxfp4_matmul_launch(const uint8_t *a, const uint8_t *as, int a_format,
                               const uint8_t *w, const uint8_t *ws, int64_t M, int64_t K,
                               int64_t N, void *Y, int type, hipStream_t stream) {
  // 33 to 64 tokens: tiles of 64x64 where there are enough of them (64x14336
  // 12.9 us, against 13.5 with 64 rows a workgroup here; fewer: 40x1056x4097
  // 6.4 against 5.9 here, 64x4128x4096 17.4 against 15.1, at the border
  // 64x4128x8192 17.7 against 18.2)
  const bool few = M <= 32 || (M <= 64 && N <= 8192);
  if (!few && K <= kMxTiledMaxDim)
    return mxfp4_matmul_tiled_launch(a, as, a_format, w, ws, M, K, N, Y, type, stream);
#define CALL(AF)                                                                        \
  switch (type) {                                                                       \
    case MX_F32: launch_rows<AF, MX_F32>(a, as, w, ws, (int)M, K, N, Y, stream); break; \
    case MX_BF16: launch_rows<AF, MX_BF16>(a, as, w, ws, (int)M, K, N, Y, stream); break; \
    default: launch_rows<AF, MX_F16>(a, as, w, ws, (int)M, K, N, Y, stream); break;     \
  }
  if (a_format == MX_FP4) { CALL(MX_FP4) } else { CALL(MX_FP8) }
#undef CALL
  return hipGetLastError();
}

}  // namespace q4k
