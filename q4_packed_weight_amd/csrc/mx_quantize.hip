// mx_quantize.hip -- rows to MX blocks and back.
#include "mx_common.h"
#include "mx_internal.h"

namespace q4k {
namespace {

constexpr int kThreads = 256;

// Each lane takes eight consecutive values of the flat array (rows are whole
// blocks, so blocks never cross a row); four neighbouring lanes hold one
// block and agree on its largest magnitude with two quad permutes: every load
// and store is of whole neighbouring lanes, nothing goes through LDS, and a
// lane's few registers leave room for enough waves to cover memory.  Bound by
// HBM: x is read once, codes and scales written once (14336x4096 fp32 to
// MXFP4, 266 MB: 37.7 us, 7.1 TB/s; one row of 4096 to MXFP8 1.9 us, a launch).
template <int T, int FMT>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const void *x, int64_t n_chunks,
                                                               uint8_t *codes, uint8_t *scales) {
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < n_chunks; c += stride) {
    float f[8];
    raw8_to_f32<T>(load_raw8<T>(x, c), f);
    const uint32_t s = mx_scale_byte<FMT>(block_amax_bits(f));
    const u32x2 q = mx_encode8<FMT>(f, s);
    if constexpr (FMT == MX_FP4) reinterpret_cast<uint32_t *>(codes)[c] = q[0];
    else reinterpret_cast<u32x2 *>(codes)[c] = q;
    if ((c & 3) == 0) scales[c >> 2] = (uint8_t)s;
  }
}

// The way back, lane for lane (14336x4096 MXFP4 to bf16, 149 MB: 21.5 us,
// 6.9 TB/s).
template <int T, int FMT, bool ONCE>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(const uint8_t *codes,
                                                                 const uint8_t *scales,
                                                                 int64_t n_chunks, void *y) {
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < n_chunks; c += stride) {
    u32x2 q = {0, 0};
    if constexpr (FMT == MX_FP4) q[0] = reinterpret_cast<const uint32_t *>(codes)[c];
    else q = reinterpret_cast<const u32x2 *>(codes)[c];
    float f[8];
    mx_decode8<FMT>(q, mx_scale_value(scales[c >> 2]), f);
    store_raw8<T, ONCE>(y, c, f32_to_raw8<T>(f));
  }
}

// A whole number of blocks of four lanes per pass: n_chunks is a multiple of
// four and so is every wave's first chunk, so a quad is active or idle as one.
int grid_for(int64_t n_chunks) {
  const int64_t g = (n_chunks + kThreads - 1) / kThreads;
  return (int)(g < (1 << 16) ? g : (1 << 16));
}

}  // namespace

#define Q4K_BY_TYPE(T_, F_, CALL)                                     \
  switch (T_) {                                                       \
    case MX_F32: if (F_ == MX_FP4) { CALL(MX_F32, MX_FP4); } else { CALL(MX_F32, MX_FP8); } break;     \
    case MX_BF16: if (F_ == MX_FP4) { CALL(MX_BF16, MX_FP4); } else { CALL(MX_BF16, MX_FP8); } break;  \
    default: if (F_ == MX_FP4) { CALL(MX_F16, MX_FP4); } else { CALL(MX_F16, MX_FP8); } break;         \
  }

hipError_t mx_quantize_launch(const void *x, int type, int format, int64_t n_rows, int64_t K,
                              uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  const int64_t n = n_rows * (K / 8);
#define CALL(T, F)                                                                         \
  hipLaunchKernelGGL((mx_quantize_kernel<T, F>), dim3(grid_for(n)), dim3(kThreads), 0,     \
                     stream, x, n, codes, scales)
  Q4K_BY_TYPE(type, format, CALL)
#undef CALL
  return hipGetLastError();
}

hipError_t mx_dequantize_launch(const uint8_t *codes, const uint8_t *scales, int format,
                                int64_t n_rows, int64_t K, void *y, int type,
                                hipStream_t stream) {
  const int64_t n = n_rows * (K / 8);
  const bool once = n * (type == MX_F32 ? 32 : 16) >= kMxOnceBytes;
#define CALL(T, F)                                                                             \
  if (once)                                                                                    \
    hipLaunchKernelGGL((mx_dequantize_kernel<T, F, true>), dim3(grid_for(n)), dim3(kThreads),  \
                       0, stream, codes, scales, n, y);                                        \
  else                                                                                         \
    hipLaunchKernelGGL((mx_dequantize_kernel<T, F, false>), dim3(grid_for(n)), dim3(kThreads), \
                       0, stream, codes, scales, n, y)
  Q4K_BY_TYPE(type, format, CALL)
#undef CALL
  return hipGetLastError();
}

}  // namespace q4k
