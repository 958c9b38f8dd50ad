// mx_internal.h -- launchers of the microscaled (MX) kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q4k {

// Values that the norm and mx_dequantize write, from this many bytes on, an
// XCD's L2, go past the caches, so that the kernel's end does not wait for them
// to be written back (the product's whole tiles do at any size): norm of
// 2048x1024 bf16 (4 MiB) 4.7 us against 5.6, of 4096x5120 30.3 against 31.5;
// 14336x4096 fp32 to MXFP4 and back to bf16 69 against 78, 1024x2048 5.6
// against 5.9.  Codes stay in cache: the product that reads them comes next.
constexpr int64_t kMxOnceBytes = (int64_t)4 << 20;

hipError_t mx_quantize_launch(const void *x, int type, int format, int64_t n_rows, int64_t K,
                              uint8_t *codes, uint8_t *scales, hipStream_t stream);
hipError_t mx_dequantize_launch(const uint8_t *codes, const uint8_t *scales, int format,
                                int64_t n_rows, int64_t K, void *y, int type, hipStream_t stream);
// format 0: no codes.
hipError_t mx_rmsnorm_launch(const void *x, const void *residual, const void *weight, float eps,
                             int type, int64_t n_rows, int64_t K, void *residual_out, void *y,
                             int format, uint8_t *codes, uint8_t *scales, hipStream_t stream);
hipError_t mxfp4_matmul_launch(const uint8_t *a, const uint8_t *as, int a_format,
                               const uint8_t *w, const uint8_t *ws, int64_t M, int64_t K,
                               int64_t N, void *Y, int type, hipStream_t stream);
// Rows of whole 128-position steps whose scales start at dwords.
inline bool mx_aligned_scales(const uint8_t *as, const uint8_t *ws, int64_t K) {
  return K % 128 == 0 && ((reinterpret_cast<uintptr_t>(as) | reinterpret_cast<uintptr_t>(ws)) & 3) == 0;
}
// The form for many tokens; K <= kMxTiledMaxDim.
constexpr int64_t kMxTiledMaxDim = (int64_t)1 << 22;
hipError_t mxfp4_matmul_tiled_launch(const uint8_t *a, const uint8_t *as, int a_format,
                                     const uint8_t *w, const uint8_t *ws, int64_t M, int64_t K,
                                     int64_t N, void *Y, int type, hipStream_t stream);

// The mixture-of-experts layer works on at most kMoeTokens tokens at a time,
// on no more than keep its logits in 32 KiB of LDS, and on no more than keep
// the parts of x and h and the slots' outputs within the 31 bits of a buffer
// view's offsets.
constexpr int kMoeTokens = 64;
constexpr int kMoeMaxLogits = 8192;
inline int64_t moe_tokens_at_once(int64_t H, int64_t F, int64_t E, int64_t k) {
  const int64_t by_logits = kMoeMaxLogits / E, widest = k * (H > F ? H : F);
  const int64_t by_view = (((int64_t)1 << 31) - 4096) / (6 * widest);
  const int64_t n = by_logits < by_view ? by_logits : by_view;
  return n < kMoeTokens ? n : kMoeTokens;
}
constexpr int kMoeMaxExperts = 256;
constexpr int kMoeMaxTopK = 16;
struct MoeArgs {
  const void *x;
  const void *router;
  const float *bias;
  const uint8_t *up, *up_s, *down, *down_s;
  void *y;
  void *workspace;
  int type, T, H, F, E, k;  // T <= moe_tokens_at_once(H, F, E, k)
};
int64_t moe_workspace_bytes(int64_t T, int64_t H, int64_t F, int64_t E, int64_t k);
hipError_t mxfp4_moe_launch(const MoeArgs &a, hipStream_t stream);

}  // namespace q4k
