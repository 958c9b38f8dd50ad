// mxfp4_matmul.hip -- products of MX activations with MXFP4 weights on the
// scaled matrix instructions.
#include <type_traits>

#include "mx_common.h"
#include "mx_internal.h"

namespace q4k {
namespace {

constexpr int kWaves = 8;

// 16 weight rows x 16 NT tokens per workgroup; its waves take the 128-position
// steps of input_dim in turn and their partial tiles are added in LDS in wave
// order.  Weights are the A operand (16 bytes a lane, as stored), activations
// the B operand; nothing is decoded.  Rows and tokens past the end read the
// last one and are not stored.
template <int AF, int T, int NT>
__global__ __launch_bounds__(kWaves * 64) void mxfp4_rows_kernel(
    const uint8_t *a, const uint8_t *as, const uint8_t *w, const uint8_t *ws, void *y, int M,
    int64_t K, int64_t N) {
  __shared__ f32x4 red[kWaves][NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t nb = K / 32, n0 = (int64_t)blockIdx.x * 16;
  const int m0 = blockIdx.y * (16 * NT);
  const int64_t row = n0 + r < N ? n0 + r : N - 1;
  const int64_t a_row_bytes = AF == MX_FP4 ? K / 2 : K;
  const uint8_t *wr = w + row * (K / 2), *wsr = ws + row * nb;
  int64_t tok[NT];
#pragma unroll
  for (int t = 0; t < NT; t++) {
    const int m = m0 + 16 * t + r;
    tok[t] = m < M ? m : M - 1;
  }
  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; t++) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int steps = (int)((nb + 3) / 4);
  for (int s = wave; s < steps; s += kWaves) {
    const int blocks = nb - 4 * (int64_t)s < 4 ? (int)(nb - 4 * (int64_t)s) : 4;
    const i32x8 wa = load_operand<MX_FP4>(wr + 64 * (int64_t)s, g, blocks);
    const int wsc = g < blocks ? wsr[4 * (int64_t)s + g] : 127;
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const i32x8 b = load_operand<AF>(a + tok[t] * a_row_bytes + (AF == MX_FP4 ? 64 : 128) * (int64_t)s,
                                       g, blocks);
      const int bs = g < blocks ? as[tok[t] * nb + 4 * (int64_t)s + g] : 127;
      acc[t] = mfma_mx<MX_FP4, AF, T == MX_F32>(wa, b, acc[t], wsc, bs);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; t++) red[wave][t][lane] = acc[t];
  __syncthreads();
  for (int t = wave; t < NT; t += kWaves) {
    f32x4 d = red[0][t][lane];
#pragma unroll
    for (int i = 1; i < kWaves; i++) d += red[i][t][lane];
    const int64_t m = m0 + 16 * t + r;
    if (m < M) {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (n0 + 4 * g + i < N) store_value<T>(y, m * N + n0 + 4 * g + i, d[i]);
    }
  }
}

template <int AF, int T>
void launch_rows(const uint8_t *a, const uint8_t *as, const uint8_t *w, const uint8_t *ws, int M,
                 int64_t K, int64_t N, void *Y, hipStream_t stream) {
  const unsigned gx = (unsigned)((N + 15) / 16);
  const auto run = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    hipLaunchKernelGGL((mxfp4_rows_kernel<AF, T, NT>), dim3(gx, (M + 16 * NT - 1) / (16 * NT)),
                       dim3(kWaves * 64), 0, stream, a, as, w, ws, Y, M, K, N);
  };
  if (M <= 16) run(std::integral_constant<int, 1>{});
  else if (M <= 32) run(std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 4>{});
}

}  // namespace

hipError_t mxfp4_matmul_launch(const uint8_t *a, const uint8_t *as, int a_format,
                               const uint8_t *w, const uint8_t *ws, int64_t M, int64_t K,
                               int64_t N, void *Y, int type, hipStream_t stream) {
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
