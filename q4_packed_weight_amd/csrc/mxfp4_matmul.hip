// mxfp4_matmul.hip -- products of MX activations with MXFP4 weights on the
// scaled matrix instructions.
#include <type_traits>

#include "mx_common.h"
#include "mx_internal.h"

namespace q4k {
namespace {

constexpr int kWaves = 8;

__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t view, uint32_t offset) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(view, (int)offset, 0, 0));
}

// Scales of the four steps from block b on: dword j's byte g is block g of
// step j.  Inside the row one load at any alignment (the lanes of a row share
// it); at the row's end a byte for each step, 127 for blocks past the end.
struct __attribute__((packed)) Packed16 { uint32_t v[4]; };
__device__ __forceinline__ void load_scales(const uint8_t *row, int64_t b, int64_t nb, int g,
                                            bool inside, int (&s)[4]) {
  if (inside) {
    const Packed16 p = *reinterpret_cast<const Packed16 *>(row + b);
#pragma unroll
    for (int j = 0; j < 4; j++) s[j] = (int)(p.v[j] >> (8 * g));
  } else {
#pragma unroll
    for (int j = 0; j < 4; j++) s[j] = b + 4 * j + g < nb ? row[b + 4 * j + g] : 127;
  }
}

// 16 NR weight rows x 16 NT tokens per workgroup, for few tokens: every wave
// takes a run of the 128-position steps of input_dim for the whole tile,
// straight from memory into operand registers (weights as the A operand,
// nothing is decoded), and the waves' partial tiles are added in LDS in wave
// order.  Bound by the weights' bytes and the latency of the first loads: D
// steps are in flight in each wave.  Rows and tokens past the end read the
// last one and are not stored; positions past the end read as zeros.
template <int AF, int T, int NR, int NT, int D>
__global__ __launch_bounds__(kWaves * 64) void mxfp4_rows_kernel(
    const uint8_t *a, const uint8_t *as, const uint8_t *w, const uint8_t *ws, void *y, int M,
    int64_t K, int64_t N) {
  __shared__ f32x4 red[kWaves][NR * NT][64];
  constexpr bool kWide = AF == MX_FP8;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t nb = K / 32, n0 = (int64_t)blockIdx.x * (16 * NR);
  const int m0 = blockIdx.y * (16 * NT);
  const int rows_n = N - n0 < 16 * NR ? (int)(N - n0) : 16 * NR;
  const int rows_m = M - m0 < 16 * NT ? M - m0 : 16 * NT;
  const uint32_t a_bytes = (uint32_t)(kWide ? K : K / 2), w_bytes = (uint32_t)(K / 2);
  const auto a_view = make_rsrc32(a + (int64_t)m0 * a_bytes, rows_m * a_bytes);
  const auto w_view = make_rsrc32(w + n0 * w_bytes, rows_n * w_bytes);

  // With an even NR the rows of two tiles are interleaved by four, so that a
  // lane ends with eight consecutive outputs.
  uint32_t w_at[NR], a_at[NT];
  const uint8_t *w_scale[NR], *a_scale[NT];
#pragma unroll
  for (int i = 0; i < NR; i++) {
    int n = 16 * i + r;
    if constexpr (NR % 2 == 0) n = (i >> 1) * 32 + (r >> 2) * 8 + (i & 1) * 4 + (r & 3);
    n = n < rows_n ? n : rows_n - 1;
    w_at[i] = (uint32_t)n * w_bytes + 16 * g;
    w_scale[i] = ws + (n0 + n) * nb;
  }
#pragma unroll
  for (int t = 0; t < NT; t++) {
    const int m = 16 * t + r < rows_m ? 16 * t + r : rows_m - 1;
    a_at[t] = (uint32_t)m * a_bytes + 16 * g;
    a_scale[t] = as + (int64_t)(m0 + m) * nb;
  }

  const int steps = (int)((nb + 3) / 4);
  const int first = (int)((int64_t)steps * wave / kWaves);
  const int last = (int)((int64_t)steps * (wave + 1) / kWaves);
  f32x4 acc[NR][NT];
#pragma unroll
  for (int i = 0; i < NR; i++)
#pragma unroll
    for (int t = 0; t < NT; t++) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  i32x4 wv[D][NR], alo[D][NT], ahi[D][NT];
  const int blocks = (int)nb;
  const auto fetch = [&](int s, int d) {
    const bool in = s < last;
    const uint32_t none = 0x7FFFFFF0u;
    const bool in_w = in && 4 * s + g < blocks;
#pragma unroll
    for (int i = 0; i < NR; i++) wv[d][i] = load16(w_view, in_w ? w_at[i] + 64u * s : none);
    if constexpr (kWide) {
      const bool in_lo = in && 4 * s + (g >> 1) < blocks, in_hi = in && 4 * s + 2 + (g >> 1) < blocks;
#pragma unroll
      for (int t = 0; t < NT; t++) {
        alo[d][t] = load16(a_view, in_lo ? a_at[t] + 128u * s : none);
        ahi[d][t] = load16(a_view, in_hi ? a_at[t] + 128u * s + 64 : none);
      }
    } else {
#pragma unroll
      for (int t = 0; t < NT; t++) alo[d][t] = load16(a_view, in_w ? a_at[t] + 64u * s : none);
    }
  };
  if (first < last) {
    int wsc[NR][4], asc[NT][4];
    const auto fetch_scales = [&](int s) {
      const bool inside = 4 * (int64_t)s + 16 <= nb;
#pragma unroll
      for (int i = 0; i < NR; i++) load_scales(w_scale[i], 4 * (int64_t)s, nb, g, inside, wsc[i]);
#pragma unroll
      for (int t = 0; t < NT; t++) load_scales(a_scale[t], 4 * (int64_t)s, nb, g, inside, asc[t]);
    };
    fetch_scales(first);
#pragma unroll
    for (int d = 0; d < D; d++) fetch(first + d, d);
    for (int s = first; s < last; s += 4) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        constexpr int kRing = D;
        const int d = j % kRing;
#pragma unroll
        for (int t = 0; t < NT; t++) {
          i32x8 b = {alo[d][t][0], alo[d][t][1], alo[d][t][2], alo[d][t][3], 0, 0, 0, 0};
          if constexpr (kWide)
            b = i32x8{alo[d][t][0], alo[d][t][1], alo[d][t][2], alo[d][t][3],
                      ahi[d][t][0], ahi[d][t][1], ahi[d][t][2], ahi[d][t][3]};
#pragma unroll
          for (int i = 0; i < NR; i++) {
            const i32x8 v = {wv[d][i][0], wv[d][i][1], wv[d][i][2], wv[d][i][3], 0, 0, 0, 0};
            acc[i][t] = mfma_mx<MX_FP4, AF, T == MX_F32>(v, b, acc[i][t], wsc[i][j], asc[t][j]);
          }
        }
        fetch(s + j + D, d);
      }
      if (s + 4 < last) fetch_scales(s + 4);
    }
  }
#pragma unroll
  for (int i = 0; i < NR; i++)
#pragma unroll
    for (int t = 0; t < NT; t++) red[wave][i * NT + t][lane] = acc[i][t];
  __syncthreads();

  typedef typename MxStore<T>::type Out;
  Out *const yo = static_cast<Out *>(y);
  const auto sum = [&](int tile) {
    f32x4 d = red[0][tile][lane];
#pragma unroll
    for (int i = 1; i < kWaves; i++) d += red[i][tile][lane];
    return d;
  };
  if constexpr (NR % 2 == 0) {
    const bool wide = N % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
    for (int q = wave; q < NR / 2 * NT; q += kWaves) {
      const int i = q / NT * 2, t = q % NT;
      const f32x4 lo = sum(i * NT + t), hi = sum((i + 1) * NT + t);
      const float f[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      const int m = 16 * t + r, n = 16 * i + 8 * g;
      if (m >= rows_m) continue;
      const int64_t at = (int64_t)(m0 + m) * N + n0 + n;
      if (wide && n + 8 <= rows_n) {
        store_raw8<T>(yo + at, 0, f32_to_raw8<T>(f));
      } else {
#pragma unroll
        for (int k = 0; k < 8; k++)
          if (n + k < rows_n) yo[at + k] = (Out)f[k];
      }
    }
  } else {
    for (int q = wave; q < NR * NT; q += kWaves) {
      const f32x4 d = sum(q);
      const int m = 16 * (q % NT) + r, n = 16 * (q / NT) + 4 * g;
      if (m >= rows_m) continue;
#pragma unroll
      for (int k = 0; k < 4; k++)
        if (n + k < rows_n) yo[(int64_t)(m0 + m) * N + n0 + n + k] = (Out)d[k];
    }
  }
}

template <int AF, int T>
void launch_rows(const uint8_t *a, const uint8_t *as, const uint8_t *w, const uint8_t *ws, int M,
                 int64_t K, int64_t N, void *Y, hipStream_t stream) {
  const auto run = [&](auto nr, auto nt, auto d) {
    constexpr int NR = decltype(nr)::value, NT = decltype(nt)::value, D = decltype(d)::value;
    hipLaunchKernelGGL((mxfp4_rows_kernel<AF, T, NR, NT, D>),
                       dim3((unsigned)((N + 16 * NR - 1) / (16 * NR)), (M + 16 * NT - 1) / (16 * NT)),
                       dim3(kWaves * 64), 0, stream, a, as, w, ws, Y, M, K, N);
  };
  typedef std::integral_constant<int, 1> One;
  typedef std::integral_constant<int, 2> Two;
  typedef std::integral_constant<int, 4> Four;
  if (M <= 16) {
    if (N <= 8192) run(One{}, One{}, Four{});
    else run(Two{}, One{}, Four{});
  } else if (M <= 32) {
    if (N <= 8192) run(One{}, Two{}, Four{});
    else run(Two{}, Two{}, Two{});
  } else {
    if (N <= 8192) run(Two{}, Four{}, Two{});
    else run(Four{}, Four{}, One{});
  }
}

}  // namespace

hipError_t mxfp4_matmul_launch(const uint8_t *a, const uint8_t *as, int a_format,
                               const uint8_t *w, const uint8_t *ws, int64_t M, int64_t K,
                               int64_t N, void *Y, int type, hipStream_t stream) {
  if (M >= 512 && N >= 512 && K <= kMxTiledMaxDim)
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
