// mx_cache.hip -- rows of keys and values to the MX blocks of a paged cache,
// and back.
#include "mx_common.h"
#include "mx_internal.h"

namespace q4k {
namespace {

constexpr int kThreads = 256;

// Eight values of a head to a lane, four lanes to a block, as mx_quantize has
// them; keys in the grid's first layer, values in its second.  Each token's
// slot is looked up by its lanes alone: nothing else depends on it, and its
// eight bytes are one line for all of them.  Bound by memory (32768 tokens of 8 heads
// of 128, bf16 to MX_FP8, 203 MB: 41 us, 5.0 TB/s), a few tokens by the launch (64: 2.6
// us).
template <int T, int FMT>
__global__ __launch_bounds__(kThreads) void mx_cache_write_kernel(CacheArgs a) {
  const bool values = blockIdx.y != 0;
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.n_chunks) return;
  const uint32_t row = a.by_chunks.of(i), c = i - row * a.chunks;
  const uint32_t t = a.by_heads.of(row), h = row - t * a.heads;
  const int64_t slot = a.slots[t];
  const typename MxStore<T>::type *const x =
      static_cast<const typename MxStore<T>::type *>(values ? a.v : a.k) +
      t * (values ? a.v_stride : a.k_stride) + (int64_t)h * a.chunks * 8;
  float f[8];
  raw8_to_f32<T>(load_raw8<T>(x, c), f);
  const uint32_t s = mx_scale_byte<FMT>(block_amax_bits(f));
  const u32x2 q = mx_encode8<FMT>(f, s);
  if ((uint64_t)slot >= (uint64_t)a.n_slots) return;
  const int64_t at = cache_row(a, slot, h) * a.chunks + c;
  uint8_t *const codes = values ? a.v_codes : a.k_codes;
  if constexpr (FMT == MX_FP4) reinterpret_cast<uint32_t *>(codes)[at] = q[0];
  else reinterpret_cast<u32x2 *>(codes)[at] = q;
  if ((c & 3) == 0) (values ? a.v_scales : a.k_scales)[at >> 2] = (uint8_t)s;
}

// The way back, lane for lane (32768 tokens of 8 heads of 128, MX_FP8 to bf16, 204
// MB: 33 us, 6.1 TB/s).
template <int T, int FMT, bool ONCE>
__global__ __launch_bounds__(kThreads) void mx_cache_read_kernel(CacheArgs a) {
  const bool values = blockIdx.y != 0;
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.n_chunks) return;
  const uint32_t row = a.by_chunks.of(i), c = i - row * a.chunks;
  const uint32_t t = a.by_heads.of(row), h = row - t * a.heads;
  const int64_t slot = a.slots[t];
  float f[8] = {};
  if ((uint64_t)slot < (uint64_t)a.n_slots) {
    const int64_t at = cache_row(a, slot, h) * a.chunks + c;
    const uint8_t *const codes = values ? a.v_codes : a.k_codes;
    u32x2 q = {0, 0};
    if constexpr (FMT == MX_FP4) q[0] = reinterpret_cast<const uint32_t *>(codes)[at];
    else q = reinterpret_cast<const u32x2 *>(codes)[at];
    mx_decode8<FMT>(q, mx_scale_value((values ? a.v_scales : a.k_scales)[at >> 2]), f);
  }
  typename MxStore<T>::type *const y =
      static_cast<typename MxStore<T>::type *>(values ? a.v_out : a.k_out) +
      t * (values ? a.v_stride : a.k_stride) + (int64_t)h * a.chunks * 8;
  store_raw8<T, ONCE>(y, c, f32_to_raw8<T>(f));
}

// Calls `go` for as many tokens at a time as a grid of 32-bit chunk numbers holds.
template <class F> hipError_t by_tokens(const CacheArgs &whole, int64_t n_tokens, size_t size, F go) {
  const int64_t per_token = (int64_t)whole.heads * whole.chunks;
  const int64_t most = ((int64_t)1 << 30) / per_token;
  for (int64_t t = 0; t < n_tokens; t += most) {
    CacheArgs a = whole;
    const int64_t n = n_tokens - t < most ? n_tokens - t : most;
    const auto in = [&](const void *p, int64_t stride) {
      return static_cast<const uint8_t *>(p) + t * stride * size;
    };
    if (a.k) a.k = in(a.k, a.k_stride), a.v = in(a.v, a.v_stride);
    if (a.k_out) {
      a.k_out = const_cast<uint8_t *>(in(a.k_out, a.k_stride));
      a.v_out = const_cast<uint8_t *>(in(a.v_out, a.v_stride));
    }
    a.slots += t;
    a.n_chunks = (uint32_t)(n * per_token);
    go(a, dim3((a.n_chunks + kThreads - 1) / kThreads, 2));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

#define Q4K_BY_TYPE(T_, F_, CALL)                                     \
  switch (T_) {                                                       \
    case MX_F32: if (F_ == MX_FP4) { CALL(MX_F32, MX_FP4); } else { CALL(MX_F32, MX_FP8); } break;     \
    case MX_BF16: if (F_ == MX_FP4) { CALL(MX_BF16, MX_FP4); } else { CALL(MX_BF16, MX_FP8); } break;  \
    default: if (F_ == MX_FP4) { CALL(MX_F16, MX_FP4); } else { CALL(MX_F16, MX_FP8); } break;         \
  }

hipError_t mx_cache_write_launch(const CacheArgs &a, int64_t n_tokens, int type, int format,
                                 hipStream_t stream) {
  return by_tokens(a, n_tokens, type == MX_F32 ? 4 : 2, [&](const CacheArgs &p, dim3 grid) {
#define CALL(T, F) \
  hipLaunchKernelGGL((mx_cache_write_kernel<T, F>), grid, dim3(kThreads), 0, stream, p)
    Q4K_BY_TYPE(type, format, CALL)
#undef CALL
  });
}

hipError_t mx_cache_read_launch(const CacheArgs &a, int64_t n_tokens, int type, int format,
                                hipStream_t stream) {
  const int64_t size = type == MX_F32 ? 4 : 2;
  const bool once = n_tokens * a.heads * a.chunks * 16 * size >= kMxOnceBytes;
  return by_tokens(a, n_tokens, size, [&](const CacheArgs &p, dim3 grid) {
#define CALL(T, F)                                                                               \
  if (once)                                                                                      \
    hipLaunchKernelGGL((mx_cache_read_kernel<T, F, true>), grid, dim3(kThreads), 0, stream, p);  \
  else                                                                                           \
    hipLaunchKernelGGL((mx_cache_read_kernel<T, F, false>), grid, dim3(kThreads), 0, stream, p)
    Q4K_BY_TYPE(type, format, CALL)
#undef CALL
  });
}

}  // namespace q4k
