// mx_rmsnorm.hip -- residual addition, root-mean-square norm, MX blocks out.
#include <algorithm>
#include <type_traits>

#include "mx_common.h"
#include "mx_internal.h"

namespace q4k {
namespace {

// Sum of one value per thread over the workgroup, in every thread: within a
// wave by cross-lane adds, then the waves' sums in order.
__device__ __forceinline__ float block_sum(float v, float *lds) {
  v = group_sum<64>(v);
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) lds[wave] = v;
  __syncthreads();
  float t = 0.0f;
  for (int i = 0; i < waves; i++) t += lds[i];
  return t;
}

// The sum the norm is taken of: x + residual rounded to the type, so that the
// next layer's residual is the vector this norm saw.
template <int T>
__device__ __forceinline__ Raw8<T> add_raw8(const Raw8<T> &a, const Raw8<T> &b) {
  float f[8], g[8];
  raw8_to_f32<T>(a, f);
  raw8_to_f32<T>(b, g);
#pragma unroll
  for (int i = 0; i < 8; i++) f[i] += g[i];
  return f32_to_raw8<T>(f);
}

template <int T>
__device__ __forceinline__ float sum_squares(const Raw8<T> &r) {
  float f[8], s = 0.0f;
  raw8_to_f32<T>(r, f);
#pragma unroll
  for (int i = 0; i < 8; i++) s = __builtin_fmaf(f[i], f[i], s);
  return s;
}

// Eight normed values: y and the codes of their block.
template <int T, bool ONCE>
__device__ __forceinline__ void emit8(const Raw8<T> &r, const Raw8<T> &w, float inv, int64_t chunk,
                                      void *y, int format, uint8_t *codes, uint8_t *scales) {
  float f[8], g[8];
  raw8_to_f32<T>(r, f);
  raw8_to_f32<T>(w, g);
#pragma unroll
  for (int i = 0; i < 8; i++) f[i] = f[i] * inv * g[i];
  if (y) store_raw8<T, ONCE>(y, chunk, f32_to_raw8<T>(f));
  if (format == MX_FP8) {
    const uint32_t s = mx_scale_byte<MX_FP8>(block_amax_bits(f));
    reinterpret_cast<u32x2 *>(codes)[chunk] = mx_encode8<MX_FP8>(f, s);
    if ((chunk & 3) == 0) scales[chunk >> 2] = (uint8_t)s;
  } else if (format == MX_FP4) {
    const uint32_t s = mx_scale_byte<MX_FP4>(block_amax_bits(f));
    reinterpret_cast<uint32_t *>(codes)[chunk] = mx_encode8<MX_FP4>(f, s)[0];
    if ((chunk & 3) == 0) scales[chunk >> 2] = (uint8_t)s;
  }
}

// One row per workgroup, held in registers as NC chunks of eight values per
// lane, so memory is read once; four neighbouring lanes hold one block.  The
// weights are sent for while the sum is made.  Bound by HBM: 4096x5120 bf16
// with residual and MXFP8 out, 147 MB, 30.2 us, 4.9 TB/s (a copy of 1 GiB
// runs at 5.2); one row of 4096 2.2 us, a launch.  The statistics are fp32:
// with fp64 sums, root and products 3 scale bytes of 63 million lay one off
// the exact ones instead of 6, at 32.9 us.
template <int T, int NC, bool ONCE>
__global__ __launch_bounds__(1024) void mx_rmsnorm_kernel(const void *x, const void *residual,
                                                          const void *weight, float eps, int n,
                                                          float inv_dim, void *residual_out,
                                                          void *y, int format,
                                                          uint8_t *codes, uint8_t *scales) {
  __shared__ float lds[16];
  const int64_t base = (int64_t)blockIdx.x * n;  // chunk index of the row's first
  Raw8<T> r[NC], w[NC];
#pragma unroll
  for (int j = 0; j < NC; j++) {
    const int c = threadIdx.x + j * blockDim.x;
    if (c < n) {
      r[j] = load_raw8<T>(x, base + c);
      if (residual) w[j] = load_raw8<T>(residual, base + c);
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < NC; j++) {
    const int c = threadIdx.x + j * blockDim.x;
    if (c < n) {
      if (residual) r[j] = add_raw8<T>(r[j], w[j]);
      ss += sum_squares<T>(r[j]);
      w[j] = load_raw8<T>(weight, c);
    }
  }
  const float inv = 1.0f / __builtin_sqrtf(block_sum(ss, lds) * inv_dim + eps);
#pragma unroll
  for (int j = 0; j < NC; j++) {
    const int c = threadIdx.x + j * blockDim.x;
    if (c < n) {
      if (residual_out) store_raw8<T, ONCE>(residual_out, base + c, r[j]);
      emit8<T, ONCE>(r[j], w[j], inv, base + c, y, format, codes, scales);
    }
  }
}

// Rows too long for registers: one pass for the sum, one for the outputs.
// Each lane writes only the chunks of residual_out that it reads again
// itself, so residual_out may be x or residual.
template <int T, bool ONCE>
__global__ __launch_bounds__(1024) void mx_rmsnorm_long_kernel(
    const void *x, const void *residual, const void *weight, float eps, int n, float inv_dim,
    void *residual_out, void *y, int format, uint8_t *codes, uint8_t *scales) {
  __shared__ float lds[16];
  const int64_t base = (int64_t)blockIdx.x * n;
  float ss = 0.0f;
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    Raw8<T> r = load_raw8<T>(x, base + c);
    if (residual) r = add_raw8<T>(r, load_raw8<T>(residual, base + c));
    ss += sum_squares<T>(r);
  }
  const float inv = 1.0f / __builtin_sqrtf(block_sum(ss, lds) * inv_dim + eps);
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    Raw8<T> r = load_raw8<T>(x, base + c);
    if (residual) r = add_raw8<T>(r, load_raw8<T>(residual, base + c));
    if (residual_out) store_raw8<T, ONCE>(residual_out, base + c, r);
    emit8<T, ONCE>(r, load_raw8<T>(weight, c), inv, base + c, y, format, codes, scales);
  }
}

}  // namespace

hipError_t mx_rmsnorm_launch(const void *x, const void *residual, const void *weight, float eps,
                             int type, int64_t n_rows, int64_t K, void *residual_out, void *y,
                             int format, uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  const int n = (int)(K / 8);
  const float inv_dim = 1.0f / (float)K;
  const bool once = n_rows * K * (type == MX_F32 ? 4 : 2) >= kMxOnceBytes;
  // chunks per lane: one up to 1024 chunks, two, then four
  const int nc = n <= 1024 ? 1 : n <= 2048 ? 2 : 4;
  const int lanes = (n + nc - 1) / nc;
  const int threads = lanes >= 1024 ? 1024 : (lanes + 63) / 64 * 64;
  const auto run = [&](auto t, auto o) {
    constexpr int T = decltype(t)::value;
    constexpr bool ONCE = decltype(o)::value;
    // A grid holds fewer than 2^32 threads, and so 2^22 rows of any block.
    constexpr int64_t kRows = ((int64_t)1 << 22) - 1;
    const auto go = [&](auto kernel, int block) {
      for (int64_t r = 0; r < n_rows; r += kRows) {
        const int64_t at = r * K, size = T == MX_F32 ? 4 : 2;
        const auto in = [&](const void *p) {
          return p ? static_cast<const uint8_t *>(p) + at * size : nullptr;
        };
        const auto out = [&](void *p) { return p ? static_cast<uint8_t *>(p) + at * size : nullptr; };
        hipLaunchKernelGGL(kernel, dim3(std::min(n_rows - r, kRows)), dim3(block), 0, stream, in(x),
                           in(residual), weight, eps, n, inv_dim, out(residual_out), out(y), format,
                           codes ? codes + at * format / 8 : nullptr,
                           scales ? scales + at / 32 : nullptr);
      }
    };
    if (n > 4096) go(mx_rmsnorm_long_kernel<T, ONCE>, 1024);
    else if (nc == 1) go(mx_rmsnorm_kernel<T, 1, ONCE>, threads);
    else if (nc == 2) go(mx_rmsnorm_kernel<T, 2, ONCE>, threads);
    else go(mx_rmsnorm_kernel<T, 4, ONCE>, threads);
  };
  const auto by_size = [&](auto t) {
    if (once) run(t, std::true_type{});
    else run(t, std::false_type{});
  };
  switch (type) {
    case MX_F32: by_size(std::integral_constant<int, MX_F32>{}); break;
    case MX_BF16: by_size(std::integral_constant<int, MX_BF16>{}); break;
    default: by_size(std::integral_constant<int, MX_F16>{}); break;
  }
  return hipGetLastError();
}

}  // namespace q4k
