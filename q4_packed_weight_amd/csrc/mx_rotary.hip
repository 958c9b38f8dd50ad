// mx_rotary.hip -- rotary positions.
#include <math.h>

#include "mx_common.h"
#include "mx_internal.h"

namespace q4k {
namespace {

constexpr int kThreads = 256;

// Cosine and sine of position * frequency.  The angle is made in turns and in
// 64 bits, and only its distance to the nearest whole turn, at most a half,
// goes on in 32: a position of 2^20 leaves 2^-33 of a turn, where 32 bits
// alone would leave none of its angle.
__device__ __forceinline__ float2 turn(int64_t position, double frequency, float amplitude) {
  const double turns = (double)position * (frequency * 0.15915494309189533577);
  const float part = (float)(turns - __builtin_rint(turns));
  float s, c;
  sincospif(2.0f * part, &s, &c);
  return make_float2(c * amplitude, s * amplitude);
}

template <int T> __device__ __forceinline__ float load_value(const void *p, int64_t i) {
  return (float)reinterpret_cast<const typename MxStore<T>::type *>(p)[i];
}

// A workgroup takes `tokens` tokens and `heads` of their heads: its lanes make
// the tokens' cosines and sines once, into LDS, and then turn whole chunks of
// eight values: two chunks half a rotary_dim apart (half layout), or one with
// four pairs (interleaved).  Without the table each head would make them again,
// and they cost more instructions than the turn.  Bound by memory for many
// tokens (4096 of 40 heads of 128, bf16, 84 MB: 17.6 us, 4.8 TB/s), by the launch for
// one (3.0 us).  x may be y: a chunk's values are read and
// written by one lane alone.
template <int T, bool HALF>
__global__ __launch_bounds__(kThreads) void mx_rotary_kernel(RotaryArgs a) {
  extern __shared__ float2 table[];
  const int pairs = a.rotary_dim / 2, t0 = (int)(blockIdx.x * a.tokens);
  const int nt = min(a.tokens, a.n_tokens - t0);
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = a.by_pairs.of(i), p = i - t * pairs;
    table[i] = turn(a.positions[t0 + t], a.frequencies[p], a.amplitude);
  }
  __syncthreads();
  const int h0 = blockIdx.y * a.heads, nh = min(a.heads, a.n_heads - h0);
  // per head: the turned chunks (pairs of chunks), then those behind rotary_dim
  const int turned = HALF ? pairs / 8 : a.rotary_dim / 8;
  const int chunks = a.chunks;  // turned + (head_dim - rotary_dim) / 8, the latter none in place
  for (int i = threadIdx.x; i < nt * a.heads * chunks; i += kThreads) {
    const int row = a.by_chunks.of(i), c = i - row * chunks;
    const int t = a.by_heads.of(row), h = row - t * a.heads;
    if (h >= nh) continue;
    const int64_t head = (int64_t)(h0 + h) * a.head_dim;
    const typename MxStore<T>::type *const x =
        static_cast<const typename MxStore<T>::type *>(a.x) + (t0 + t) * a.x_stride + head;
    typename MxStore<T>::type *const y =
        static_cast<typename MxStore<T>::type *>(a.y) + (t0 + t) * a.y_stride + head;
    const float2 *const cs = table + t * pairs;
    if (c >= turned) {
      const int at = a.rotary_dim / 8 + c - turned;
      store_raw8<T>(y, at, load_raw8<T>(x, at));
    } else if constexpr (HALF) {
      float f[8], g[8];
      raw8_to_f32<T>(load_raw8<T>(x, c), f);
      raw8_to_f32<T>(load_raw8<T>(x, c + turned), g);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float2 w = cs[8 * c + j];
        const float v = f[j] * w.x - g[j] * w.y;
        g[j] = g[j] * w.x + f[j] * w.y;
        f[j] = v;
      }
      store_raw8<T>(y, c, f32_to_raw8<T>(f));
      store_raw8<T>(y, c + turned, f32_to_raw8<T>(g));
    } else {
      float f[8];
      raw8_to_f32<T>(load_raw8<T>(x, c), f);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float2 w = cs[4 * c + j];
        const float v = f[2 * j] * w.x - f[2 * j + 1] * w.y;
        f[2 * j + 1] = f[2 * j + 1] * w.x + f[2 * j] * w.y;
        f[2 * j] = v;
      }
      store_raw8<T>(y, c, f32_to_raw8<T>(f));
    }
  }
}

// The same by single pairs and values, where rotary_dim is not made of whole
// chunks.
template <int T, bool HALF>
__global__ __launch_bounds__(kThreads) void mx_rotary_pairs_kernel(RotaryArgs a) {
  extern __shared__ float2 table[];
  const int pairs = a.rotary_dim / 2, t0 = (int)(blockIdx.x * a.tokens);
  const int nt = min(a.tokens, a.n_tokens - t0);
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = a.by_pairs.of(i), p = i - t * pairs;
    table[i] = turn(a.positions[t0 + t], a.frequencies[p], a.amplitude);
  }
  __syncthreads();
  const int h0 = blockIdx.y * a.heads, nh = min(a.heads, a.n_heads - h0);
  const int items = a.chunks;  // pairs, then the values behind rotary_dim
  for (int i = threadIdx.x; i < nt * a.heads * items; i += kThreads) {
    const int row = a.by_chunks.of(i), c = i - row * items;
    const int t = a.by_heads.of(row), h = row - t * a.heads;
    if (h >= nh) continue;
    const int64_t head = (int64_t)(h0 + h) * a.head_dim;
    const int64_t xr = (t0 + t) * a.x_stride + head, yr = (t0 + t) * a.y_stride + head;
    if (c >= pairs) {
      const int at = a.rotary_dim + c - pairs;
      store_value<T>(a.y, yr + at, load_value<T>(a.x, xr + at));
    } else {
      const int one = HALF ? c : 2 * c, two = HALF ? c + pairs : 2 * c + 1;
      const float2 w = table[t * pairs + c];
      const float f = load_value<T>(a.x, xr + one), g = load_value<T>(a.x, xr + two);
      store_value<T>(a.y, yr + one, f * w.x - g * w.y);
      store_value<T>(a.y, yr + two, g * w.x + f * w.y);
    }
  }
}

}  // namespace

hipError_t mx_rotary_launch(const void *x, int64_t x_stride, int type, const int64_t *positions,
                            const double *frequencies, float amplitude, int64_t n_tokens,
                            int n_heads, int head_dim, int rotary_dim, bool half, void *y,
                            int64_t y_stride, hipStream_t stream) {
  RotaryArgs a;
  a.positions = positions;
  a.frequencies = frequencies;
  a.amplitude = amplitude;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.n_heads = n_heads;
  a.head_dim = head_dim;
  a.rotary_dim = rotary_dim;
  const bool in_place = x == y && x_stride == y_stride;
  const bool whole = rotary_dim % (half ? 16 : 8) == 0;
  const int pairs = rotary_dim / 2, rest = in_place ? 0 : head_dim - rotary_dim;
  a.chunks = whole ? (half ? pairs / 8 : rotary_dim / 8) + rest / 8 : pairs + rest;
  if (a.chunks == 0) a.chunks = 1;
  // Tokens of a workgroup: enough for a cosine and sine a lane; heads: all of
  // them, unless too few workgroups would come out.
  a.tokens = pairs >= kThreads ? 1 : kThreads / pairs;
  a.heads = n_heads;
  const int64_t enough = 512;
  while (a.tokens > 1 && (n_tokens + a.tokens - 1) / a.tokens < enough) a.tokens = (a.tokens + 1) / 2;
  const int64_t groups = (n_tokens + a.tokens - 1) / a.tokens;
  while (a.heads > 1 && groups * ((n_heads + a.heads - 1) / a.heads) < enough &&
         a.tokens * a.heads * a.chunks > kThreads)
    a.heads = (a.heads + 1) / 2;
  a.by_pairs = FastDiv(pairs);
  a.by_chunks = FastDiv(a.chunks);
  a.by_heads = FastDiv(a.heads);
  const size_t size = type == MX_F32 ? 4 : 2;
  // a grid holds fewer than 2^32 threads
  const int64_t rows = (((int64_t)1 << 23) / ((n_heads + a.heads - 1) / a.heads)) * a.tokens;
  for (int64_t t = 0; t < n_tokens; t += rows) {
    a.x = static_cast<const uint8_t *>(x) + t * x_stride * size;
    a.y = static_cast<uint8_t *>(y) + t * y_stride * size;
    a.positions = positions + t;
    a.n_tokens = (int)(n_tokens - t < rows ? n_tokens - t : rows);
    const dim3 grid((a.n_tokens + a.tokens - 1) / a.tokens, (n_heads + a.heads - 1) / a.heads);
    const size_t lds = (size_t)a.tokens * pairs * sizeof(float2);
#define GO(K, T)                                                                       \
  do {                                                                                 \
    if (half) hipLaunchKernelGGL((K<T, true>), grid, dim3(kThreads), lds, stream, a);  \
    else hipLaunchKernelGGL((K<T, false>), grid, dim3(kThreads), lds, stream, a);      \
  } while (0)
#define BY_TYPE(K)                          \
  switch (type) {                           \
    case MX_F32: GO(K, MX_F32); break;      \
    case MX_BF16: GO(K, MX_BF16); break;    \
    default: GO(K, MX_F16); break;          \
  }
    if (whole) {
      BY_TYPE(mx_rotary_kernel)
    } else {
      BY_TYPE(mx_rotary_pairs_kernel)
    }
#undef BY_TYPE
#undef GO
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

void mx_rotary_frequencies_make(int d, double base, int scaling, double factor, double trained,
                                double low, double high, double *f, double *amplitude) {
  const double pi2 = 6.283185307179586476925;
  *amplitude = 1.0;
  if (scaling == MX_ROTARY_NTK && d > 2) base *= pow(factor, (double)d / (d - 2));
  // the index (not a whole one) of the pair that turns `turns` times over the trained context
  const auto at = [&](double turns) { return d * log(trained / (turns * pi2)) / (2 * log(base)); };
  double first = 0, last = 0;
  if (scaling == MX_ROTARY_YARN) {
    first = fmax(floor(at(high)), 0.0);
    last = fmin(ceil(at(low)), d - 1.0);
    *amplitude = 0.1 * log(factor) + 1.0;
  }
  for (int i = 0; i < d / 2; i++) {
    const double x = pow(base, -2.0 * i / d);
    double keep = 1.0;  // the share of the unscaled frequency
    if (scaling == MX_ROTARY_LINEAR) keep = 0.0;
    if (scaling == MX_ROTARY_YARN) keep = 1.0 - fmin(1.0, fmax(0.0, (i - first) / fmax(last - first, 1e-3)));
    if (scaling == MX_ROTARY_BANDS) keep = fmin(1.0, fmax(0.0, (trained * x / pi2 - low) / (high - low)));
    f[i] = x * (keep + (1.0 - keep) / factor);
  }
}

}  // namespace q4k
