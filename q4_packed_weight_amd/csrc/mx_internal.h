// mx_internal.h -- launchers of the microscaled (MX) kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4k_mx.h"

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

// Division of 0 <= n < 2^31 by d: n * m >> shift with m = floor(2^shift / d) + 1
// and shift = 31 + ceil(log2 d), whose excess over n / d stays below 1 / d.
struct FastDiv {
  uint32_t m = 0, shift = 0;
  FastDiv() = default;
  explicit FastDiv(uint32_t d) {
    uint32_t l = 0;
    while (((uint64_t)1 << l) < d) l++;
    shift = 31 + l;
    m = (uint32_t)(((uint64_t)1 << shift) / d + 1);
  }
  __host__ __device__ uint32_t of(uint32_t n) const { return (uint32_t)((uint64_t)n * m >> shift); }
};

struct RotaryArgs {
  const void *x;
  void *y;
  const int64_t *positions;
  const double *frequencies;
  int64_t x_stride, y_stride;  // values from a token's row to the next
  float amplitude;
  int n_tokens, n_heads, head_dim, rotary_dim;
  int tokens, heads, chunks;  // of a workgroup; chunks of a head
  FastDiv by_pairs, by_chunks, by_heads;
};
hipError_t mx_rotary_launch(const void *x, int64_t x_stride, int type, const int64_t *positions,
                            const double *frequencies, float amplitude, int64_t n_tokens,
                            int n_heads, int head_dim, int rotary_dim, bool half, void *y,
                            int64_t y_stride, hipStream_t stream);
void mx_rotary_frequencies_make(int d, double base, int scaling, double factor, double trained,
                                double low, double high, double *f, double *amplitude);

// A paged cache: row (page * heads + head) * page_size + place of each array.
struct CacheArgs {
  const void *k, *v;    // of mx_cache_write
  void *k_out, *v_out;  // of mx_cache_read
  int64_t k_stride, v_stride;
  const int64_t *slots;
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int64_t n_slots;
  uint32_t n_chunks;       // of this launch, each of keys and values
  uint32_t heads, chunks;  // chunks of eight values of a head
  uint32_t page_size;
  FastDiv by_chunks, by_heads, by_page;
};
__device__ __forceinline__ int64_t cache_row(const CacheArgs &a, int64_t slot, uint32_t head) {
  const uint32_t page = a.by_page.of((uint32_t)slot), place = (uint32_t)slot - page * a.page_size;
  return ((int64_t)page * a.heads + head) * a.page_size + place;
}
hipError_t mx_cache_write_launch(const CacheArgs &a, int64_t n_tokens, int type, int format,
                                 hipStream_t stream);
hipError_t mx_cache_read_launch(const CacheArgs &a, int64_t n_tokens, int type, int format,
                                hipStream_t stream);

struct AttentionArgs {
  const void *q;
  void *y;
  int64_t q_stride, y_stride;
  const int32_t *starts, *counts, *table;
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  float *partial;   // [n_parts][head_dim], then [n_parts][2]
  int64_t n_parts;  // rows of partial results
  int type, format, n_tokens, n_heads, n_kv_heads, group, head_dim;
  int n_seqs, pages_per_seq, max_queries, n_pages, page_size;
  int causal, window;  // window 0: none
  // tiles of rows that a sequence has at most; where `planned`, workgroups find
  // their sequence by its sizes, and cut the keys into shares for about
  // shares_wanted (0: none) of them a key head; units they are at most
  int tiles, planned, shares_wanted, units;
  float scale;         // times log2(e), without its power of two: +-[0.5, 1), or 0
  int scale_power;
  FastDiv by_page, by_group, by_kv_heads, by_tiles;
};
// Sizes alone decide the launch: the same call has the same workspace.
int64_t mx_attention_workspace_bytes(AttentionArgs &a);
hipError_t mx_attention_launch(const AttentionArgs &a, hipStream_t stream);

}  // namespace q4k
