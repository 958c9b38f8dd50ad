// mxfp4_moe.hip -- a mixture-of-experts layer of MXFP4 weights for a few
// tokens, as three kernels: the router's logits, the gate and up products
// with the activation between them, and the down product with the sum over
// the chosen experts.
//
// An expert's weights are read once for up to 16 of its tokens, again for the
// next ones, and again for each 64 tokens of the call; everything else is
// small, so for few tokens the layer is bound by the weight stream (2 of 8
// experts of 4096x14336 bf16: 32 tokens 192 us; 64 tokens, about 1.4 passes,
// 290; 256 tokens 1142, 1024 tokens 4641).  e2m1 codes times their block's power
// of two are exact bf16 values, made by one conversion instruction a pair,
// and run on the 16x16x32 bf16 matrix instruction as its A operand (16 rows);
// tokens are the columns.  Activations that bf16 cannot hold enter as the sum
// of two or three bf16 values, one product each.
#include <algorithm>
#include <type_traits>

#include "mx_internal.h"
#include "mx_lds.h"

namespace q4k {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kCoherent = 16;  // sc1: the agent-coherent cache policy

// v as a sum of NP bf16 values, each the nearest to what the ones before it
// leave: 8, 16 or 24 significant bits.
template <int NP> __device__ __forceinline__ void split_bf16(float v, __bf16 (&p)[NP]) {
#pragma unroll
  for (int i = 0; i < NP; i++) {
    p[i] = (__bf16)v;
    v -= (float)p[i];
  }
}

// The order of logits as unsigned integers from 1 on: NaN lowest, -0 equal
// to +0.
__device__ __forceinline__ uint32_t logit_key(float l) {
  if (l != l) return 1u;
  const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Workspace of up to kMoeTokens tokens.
struct Workspace {
  float *logits;        // [T][E]
  int *work;            // [groups] an expert and its number of tokens << 16
  int *slots;           // [groups][kMoeTokens] their slots: token * k + rank
  float *chosen_logit;  // [T*k]
  unsigned *arrived;    // [H/16] workgroups of the down product that are done
  __bf16 *xp;           // [NPX][T][H] x in bf16 parts, none for bf16 x
  __bf16 *hp;           // [NPH][T*k][F] h in bf16 parts
  float *out;           // [T*k][H] the down product by slot
  int64_t bytes;
};

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// Parts of x and of h: h carries fp32 sums, of which two parts keep 16 bits
// (below a 16-bit output's rounding), three 24.
template <int T> constexpr int kXParts = T == MX_BF16 ? 1 : T == MX_F16 ? 2 : 3;
template <int T> constexpr int kHParts = T == MX_F32 ? 3 : 2;

Workspace layout(void *base, int type, int64_t T, int64_t H, int64_t F, int64_t E, int64_t k) {
  const int64_t px = type == MX_F32 ? 3 : 2, ph = type == MX_F32 ? 3 : 2;
  char *p = static_cast<char *>(base);
  Workspace w;
  int64_t o = 0;
  const auto take = [&](int64_t n) {
    char *const at = p + o;
    o += align256(n);
    return at;
  };
  w.logits = reinterpret_cast<float *>(take(T * E * 4));
  w.work = reinterpret_cast<int *>(take(E * 4));
  w.slots = reinterpret_cast<int *>(take(E * kMoeTokens * 4));
  w.chosen_logit = reinterpret_cast<float *>(take(T * k * 4));
  w.arrived = reinterpret_cast<unsigned *>(take(H / 16 * 4));
  w.xp = reinterpret_cast<__bf16 *>(take(px * T * H * 2));
  w.hp = reinterpret_cast<__bf16 *>(take(ph * T * k * F * 2));
  w.out = reinterpret_cast<float *>(take(T * k * H * 4));
  w.bytes = o;
  return w;
}

// logits[t, e] for TT tokens per workgroup and one expert; the workgroups
// also share out the splitting of x, and the down product's counters start
// from zero here.  Bound by latency: 2.4 us for one token, 4.6 for 13 of 1056
// on 24 experts.
template <int TY, int TT>
__global__ __launch_bounds__(256) void moe_router_kernel(const void *x, const void *router,
                                                         const float *bias, float *logits,
                                                         __bf16 *xp, unsigned *arrived, int T,
                                                         int H, int E) {
  __shared__ float lds[4][TT];
  const int e = blockIdx.x, t0 = blockIdx.y * TT, chunks = H / 8;
  float acc[TT];
#pragma unroll
  for (int t = 0; t < TT; t++) acc[t] = 0.0f;
  for (int c = threadIdx.x; c < chunks; c += 256) {
    float w[8];
    raw8_to_f32<TY>(load_raw8<TY>(router, (int64_t)e * chunks + c), w);
#pragma unroll
    for (int t = 0; t < TT; t++) {
      const int tok = t0 + t < T ? t0 + t : T - 1;
      float f[8];
      raw8_to_f32<TY>(load_raw8<TY>(x, (int64_t)tok * chunks + c), f);
#pragma unroll
      for (int i = 0; i < 8; i++) acc[t] = __builtin_fmaf(w[i], f[i], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < TT; t++) {
    const float s = group_sum<64>(acc[t]);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6][t] = s;
  }
  __syncthreads();
  if (threadIdx.x < TT && t0 + (int)threadIdx.x < T) {
    const int t = threadIdx.x;
    float s = (lds[0][t] + lds[1][t]) + (lds[2][t] + lds[3][t]);
    if (bias) s += bias[e];
    logits[(int64_t)(t0 + t) * E + e] = s;
  }
  for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x; i < H / 16;
       i += gridDim.x * gridDim.y * 256)
    arrived[i] = 0;
  constexpr int NP = kXParts<TY>;
  if constexpr (NP > 1) {
    const int64_t n = (int64_t)T * chunks;
    const int64_t stride = (int64_t)gridDim.x * gridDim.y * 256;
    for (int64_t c = (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x; c < n;
         c += stride) {
      float f[8];
      raw8_to_f32<TY>(load_raw8<TY>(x, c), f);
      bf16x8 part[NP];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        __bf16 p[NP];
        split_bf16<NP>(f[i], p);
#pragma unroll
        for (int q = 0; q < NP; q++) part[q][i] = p[q];
      }
#pragma unroll
      for (int q = 0; q < NP; q++) reinterpret_cast<bf16x8 *>(xp)[q * n + c] = part[q];
    }
  }
}

// A lane's 32 codes of one block as four bf16 operands of eight.
__device__ __forceinline__ void decode_block(i32x4 c, uint32_t s, bf16x8 (&a)[4]) {
  // 2^(s-127) from its exponent field alone: the conversion reads no more of
  // its scale, and every code comes out exact, down to s = 0 and NaN at 255
  const float scale = __builtin_bit_cast(float, s << 23);
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)c[j], scale, 0);
    const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)c[j], scale, 1);
    const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)c[j], scale, 2);
    const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)c[j], scale, 3);
    a[j] = bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
  }
}

// What a workgroup's waves multiply: V views of up to NRV tiles of 16 weight
// rows each, and 4 XC columns of activations in NP bf16 parts.  Weights come
// two steps of 128 positions at a time, 128 bytes of a row: half that, a
// step's, is half a cache line, and ran at 0.87 of the speed (499 MB of gate
// and up rows, loads alone: 121 against 105 us).
template <int V> struct Rows {
  i32x4 codes[V], scales[V];  // views of the tiles' rows
  const uint8_t *scale_base[V];
  int rows;                   // of each view, a multiple of 16
  uint32_t row_bytes;
};

// `rows` rows of a matrix of input_dim K.
template <int V>
__device__ __forceinline__ void set_rows(Rows<V> &w, int v, const uint8_t *codes,
                                         const uint8_t *scales, int rows, int64_t K) {
  w.rows = rows;
  w.row_bytes = (uint32_t)(K / 2);
  w.codes[v] = buffer_view(codes, (uint32_t)rows * w.row_bytes);
  w.scales[v] = buffer_view(scales, (uint32_t)rows * (uint32_t)(K / 32));
  w.scale_base[v] = scales;
}

template <int XC> struct Columns {  // 4 XC of them
  i32x4 view;
  uint32_t at[XC], part_bytes;    // this lane's bytes of its row of each load
};

// The columns: `source(i)` is the row of the activations [..][K] of column i,
// negative for none.  A step's 128 positions of a column are 256 bytes, in 16
// chunks of eight values; chunk c is kept at place c ^ (column % 8), so that
// an operand read of eight columns lies on all banks.
template <int XC, class F>
__device__ __forceinline__ void set_columns(Columns<XC> &x, F source, int64_t K) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < XC; i++) {
    const int column = 4 * i + (lane >> 4), chunk = (lane & 15) ^ (column & 7);
    const int row = source(column);
    x.at[i] = row < 0 ? kPastEnd : (uint32_t)row * (uint32_t)(2 * K) + 16 * chunk;
  }
}

// The products of steps first .. last-1 of one wave (first a multiple of P),
// through rings of its own in LDS at `xring` and `ring` (no barrier): SX steps
// of activations, which come from cache, SW units of P steps of weights, which
// come from memory, and the scales of four steps.  ALIGNED: rows of whole
// steps whose scales start at dwords; others come through registers, whose
// wait also waits for what is in flight.  The first units' weights are sent
// for before `columns(x)` says where the activations are, or that there are
// none (false, which is the result then).
// P = 2 takes 128 bytes of a row at a time, a cache line, and P = 1 half of
// it, which long rows feel (the loads alone of 499 MB of gate and up rows of
// 4096: 121 against 105 us); but a ring of two pairs leaves less room for wide
// tiles (32 tokens on 4 of 32 experts of 2880x2880 fp16, up: 103 us with
// P = 1, 124 with P = 2).  Whole lines are not kept in cache, half lines are
// until their other half is taken.
template <int V, int NRV, int XC, int NP, int P, int SW, int SX> struct MoeRing {
  static constexpr int kTiles = V * NRV, kX = XC * NP * 1024, kUnit = kTiles * P * 1024;
  static constexpr int kColumns = SX * kX;                                 // a wave's activations
  static constexpr int kScales = SW * kUnit, kBytes = kScales + V * 1024;  // its weights, scales
  static_assert((SX == 2 || SX == 3) && SW >= 2 && (P == 1 || P == 2) && NRV <= 4, "");
  static_assert(P == 2 || SX == 2 || SW == 3, "the waits below");
};
template <int V, int NRV, int XC, int NP, int P, int SW, int SX, bool ALIGNED, class F>
__device__ __forceinline__ bool moe_stream(uint8_t *xring, uint8_t *ring, const Rows<V> &w,
                                           Columns<XC> &x, F columns, int nb, int first,
                                           int last, f32x4 (&acc)[V * NRV]) {
  typedef MoeRing<V, NRV, XC, NP, P, SW, SX> R;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const uint32_t to_ring = lds_address(ring), to_xring = lds_address(xring);
  uint8_t *const scales = ring + R::kScales;
#pragma unroll
  for (int i = 0; i < R::kTiles; i++) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // In LDS a tile's step is an MX_FP4 tile (one load of 16 rows x 64 bytes), a
  // pair of steps lies as an MX_FP8 tile does (two loads of 8 rows x 128).
  constexpr int kForm = P == 2 ? MX_FP8 : MX_FP4;
  const int w_chunk = tile_chunk<kForm>(lane);
  const uint32_t w_at = (uint32_t)tile_row<kForm>(lane) * w.row_bytes + 16 * w_chunk;
  const auto issue_w = [&](int s, int buf) {
    const uint32_t to = to_ring + buf * R::kUnit;
    const bool in = (ALIGNED && P == 1) || 4 * s + w_chunk < nb;
#pragma unroll
    for (int i = 0; i < R::kTiles; i++)
#pragma unroll
      for (int h = 0; h < P; h++) {
        const int row = 16 * (i % NRV) + 8 * h;
        load16_to_lds<P == 2>(
            w.codes[i / NRV],
            in && row < w.rows ? w_at + (uint32_t)row * w.row_bytes + 64u * s : kPastEnd,
            to + (P * i + h) * 1024);
      }
  };
  const auto issue_x = [&](int s, int buf) {
    const uint32_t to = to_xring + buf * R::kX;
#pragma unroll
    for (int i = 0; i < XC; i++) {
      const int chunk = (lane & 15) ^ ((4 * i + (lane >> 4)) & 7);
      const bool in_x = ALIGNED || 4 * s + (chunk >> 2) < nb;
#pragma unroll
      for (int q = 0; q < NP; q++)
        load16_to_lds(x.view, in_x ? x.at[i] + q * x.part_bytes + 256u * s : kPastEnd,
                      to + (XC * q + i) * 1024);
    }
  };
  // scales: row `lane` of each view
  u32x4 held[V];
  const bool has_row = lane < 16 * NRV && lane < w.rows;
  const uint32_t scale_at = (uint32_t)(lane * nb);
  const auto load_scales = [&](int s) {
#pragma unroll
    for (int v = 0; v < V; v++)
      if (has_row) held[v] = load_scales16(w.scale_base[v] + scale_at, 4 * s, nb);
  };
  const auto issue_scales = [&](int s) {
#pragma unroll
    for (int v = 0; v < V; v++)
      load16_to_lds(w.scales[v], has_row ? scale_at + 4u * s : kPastEnd,
                    to_ring + R::kScales + v * 1024);
  };
  const int units = (last - first + P - 1) / P;
  if (first < last) {
    if constexpr (ALIGNED) issue_scales(first);
    else load_scales(first);
  }
#pragma unroll
  for (int d = 0; d < SW - 1; d++)
    if (d < units) issue_w(first + P * d, d);
  if (!columns(x)) {
    wait_loads<0>();
    return false;
  }
  if (first >= last) return true;
#pragma unroll
  for (int d = 0; d < SX - 1; d++)
    if (first + d < last) issue_x(first + d, d);
  int buf = 0, xbuf = 0;
  uint32_t sc[R::kTiles];
  // Not unrolled: a workgroup runs few steps, and code that is fetched for
  // one use costs more than the loop.
#pragma unroll 1
  for (int s = first; s < last; s++) {
    const int i = s - first, j4 = i & 3;  // j4: of the four steps whose scales are at hand
    wait_lds();                           // what the next loads overwrite is read
    const bool more_w = i / P + SW - 1 < units, more_x = s + SX - 1 < last;
    if (i % P == 0 && more_w) issue_w(s + P * (SW - 1), buf == 0 ? SW - 1 : buf - 1);
    if (more_x) issue_x(s + SX - 1, xbuf == 0 ? SX - 1 : xbuf - 1);
    if (j4 == 1 && s + 3 < last) {
      if constexpr (ALIGNED) issue_scales(s + 3);
      else load_scales(s + 3);
    }
    // Until step s's activations are there, sent SX - 1 steps ago; its weights
    // and its scales are older.  Younger: the activations of the steps since,
    // the weights sent in these steps, the next scales until they are needed.
    const int young_x = more_x ? SX - 1 : last - 1 - s;
    int young_w = (P == 1 || SX == 3 || i % P == 0) && more_w;
    if (P == 1 && SX == 3) young_w += i > 0 && (i - 1) / P + SW - 1 < units;
    const bool young_scales = ALIGNED && j4 >= 1 && j4 <= SX && s - j4 + 4 < last;
    const auto wait = [&](auto nx, auto nw) {
      constexpr int n = decltype(nx)::value * XC * NP + decltype(nw)::value * R::kTiles * P;
      if (young_scales) wait_loads<n + V>();
      else wait_loads<n>();
    };
    const auto wait_w = [&](auto nx) {
      if (P == 1 && SX == 3 && young_w == 2)
        wait(nx, std::integral_constant<int, (P == 1 && SX == 3 ? 2 : 0)>{});
      else if (young_w) wait(nx, std::integral_constant<int, 1>{});
      else wait(nx, std::integral_constant<int, 0>{});
    };
    if (SX == 3 && young_x == 2) wait_w(std::integral_constant<int, (SX == 3 ? 2 : 0)>{});
    else if (young_x) wait_w(std::integral_constant<int, 1>{});
    else wait_w(std::integral_constant<int, 0>{});
    if (j4 == 0) {
      if constexpr (!ALIGNED) {
#pragma unroll
        for (int v = 0; v < V; v++)
          if (has_row) *reinterpret_cast<u32x4 *>(scales + v * 1024 + lane * 16) = held[v];
        wait_lds();
      }
      const uint32_t which = byte_of_two(g);
#pragma unroll
      for (int t = 0; t < R::kTiles; t++)
        sc[t] = byte_of_four(*reinterpret_cast<const u32x4 *>(scales + t / NRV * 1024 +
                                                              t % NRV * 256 + r * 16), which);
    }
    const uint8_t *xs = xring + xbuf * R::kX, *ws = ring + buf * R::kUnit;
    const int column = XC == 4 ? r : r % (4 * XC);  // the others' results are not used
    bf16x8 b[NP][4];
#pragma unroll
    for (int q = 0; q < NP; q++)
#pragma unroll
      for (int j = 0; j < 4; j++)
        b[q][j] = *reinterpret_cast<const bf16x8 *>(xs + q * (XC * 1024) + column * 256 +
                                                    16 * ((4 * g + j) ^ (column & 7)));
    const int at = operand_at<kForm>(r, g) ^ (P == 2 ? 64 * (i & 1) : 0);
#pragma unroll
    for (int t = 0; t < R::kTiles; t++) {
      bf16x8 a[4];
      decode_block(*reinterpret_cast<const i32x4 *>(ws + t * (P * 1024) + at), (sc[t] >> (8 * j4)) & 255u,
                   a);
#pragma unroll
      for (int q = 0; q < NP; q++)
#pragma unroll
        for (int j = 0; j < 4; j++)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], b[q][j], acc[t], 0, 0, 0);
    }
    if (i % P == P - 1) buf = buf == SW - 1 ? 0 : buf + 1;
    xbuf = xbuf == SX - 1 ? 0 : xbuf + 1;
  }
  wait_lds();
  return true;
}

// A wave's steps: whole units of P, as even as they come.
struct Steps { int first, last; };
template <int P> __device__ __forceinline__ Steps steps_of(int nb, int wave, int waves) {
  const int steps = (nb + 3) / 4, units = (steps + P - 1) / P;
  const int first = P * (units * wave / waves), last = P * (units * (wave + 1) / waves);
  return {first, last < steps ? last : steps};
}

// The waves' sums of tile i, in wave order, from where moe_stream's rings
// were (kept there by keep_sums; a barrier between the two).
template <int TILES>
__device__ __forceinline__ void keep_sums(uint8_t *ring, const f32x4 (&acc)[TILES]) {
#pragma unroll
  for (int i = 0; i < TILES; i++)
    *reinterpret_cast<f32x4 *>(ring + i * 1024 + (threadIdx.x & 63) * 16) = acc[i];
}
template <int W> __device__ __forceinline__ f32x4 sum_of(const uint8_t *rings, int bytes, int i) {
  const uint8_t *p = rings + i * 1024 + (threadIdx.x & 63) * 16;
  f32x4 d = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
  for (int w = 1; w < W; w++) d += *reinterpret_cast<const f32x4 *>(p + w * bytes);
  return d;
}

struct UpArgs {
  const __bf16 *xp;
  const float *logits;
  const uint8_t *up, *up_s;
  int *work, *slots;
  float *chosen_logit;
  __bf16 *hp;
  int T, H, F, E, k;
  int by_slot;  // blockIdx.y is a slot, else an expert
};

// The dwords from one token's keys to the next one's in LDS: whole 16 bytes,
// and not a multiple of all banks.
__host__ __device__ inline int key_stride(int E) { return (E + 3) / 4 * 4 + 4; }

// How many of the experts from..to-1 (multiples of 4; keys past the last
// expert are 0) come before expert q: a greater key, or the same one at a
// lower index.  Whole quads before q's take keys of mine on, those after it
// greater ones; only q's own quad looks at its places.
__device__ __forceinline__ int count_before(const uint32_t *row, int from, int to, int q) {
  const uint32_t mine = row[q];
  const int own = q & ~3;
  int before = 0;
#pragma unroll 4
  for (int i = from; i < to; i += 4) {
    const u32x4 v = *reinterpret_cast<const u32x4 *>(row + i);
    const uint32_t least = i < own ? mine - 1 : mine;
#pragma unroll
    for (int c = 0; c < 4; c++) before += v[c] > least;
  }
  if (own >= from && own < to) {
    const u32x4 v = *reinterpret_cast<const u32x4 *>(row + own);
#pragma unroll
    for (int c = 0; c < 3; c++) before += own + c < q && v[c] == mine;
  }
  return before;
}

// Gate and up rows of 16 NF positions of one expert for every token that
// chose it, 4 XC tokens at a time.  An expert's rank for a token is the number
// of experts before it in the order (logit descending, index ascending), so
// each workgroup finds its tokens by counting, without a sort; ranks below k
// are the chosen ones and give each slot exactly one writer.  Bound by the
// weights (32 tokens on 2 of 8 experts of 4096x14336: 499 MB in 116 us, 4.3
// TB/s; a copy runs at 5.2), for one token by the router's latency before it,
// its own prologue (about 2 us) and the first load (8.5 us, 17.8 MB).
template <int NPX, int NPH, int NF, int XC, int W, int P, int SW, int SX, bool ALIGNED>
__global__ __launch_bounds__(W * 64) void moe_up_kernel(UpArgs p) {
  typedef MoeRing<2, NF, XC, NPX, P, SW, SX> Ring;
  constexpr int kThreads = W * 64;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[W * Ring::kBytes];
  // the logits' keys [T][key_stride(E)] first, the waves' activations later
  extern __shared__ __attribute__((aligned(1024))) uint8_t shared_lds[];
  uint32_t *const keys = reinterpret_cast<uint32_t *>(shared_lds);
  __shared__ int rank_of[kMoeTokens];
  __shared__ int list[kMoeTokens];  // token | rank << 8
  __shared__ int found, list_n;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int stride = key_stride(p.E), padded = stride - 4;
  // eight tokens' logits in flight at a time
  for (int t0 = wave; t0 < p.T; t0 += 8 * W)
    for (int q = lane; q < padded; q += 64) {
      float l[8];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int t = t0 + j * W;
        l[j] = t < p.T && q < p.E ? p.logits[t * p.E + q] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (t0 + j * W < p.T)
          keys[(t0 + j * W) * stride + q] = q < p.E ? logit_key(l[j]) : 0u;
    }
  if (tid < kMoeTokens) rank_of[tid] = 0;
  lds_barrier();
  int e = blockIdx.y, t_first = -1;
  if (p.by_slot) {
    t_first = blockIdx.y / p.k;
    const int rank = blockIdx.y % p.k;
    const uint32_t *row = keys + t_first * stride;
    for (int q = tid; q < p.E; q += kThreads)
      if (count_before(row, 0, padded, q) == rank) found = q;
    lds_barrier();
    e = __builtin_amdgcn_readfirstlane(found);
  }
  // tokens on lanes, a wave's share of the experts each
  const auto find_tokens = [&]() {
    if (p.T == 1) {  // by_slot: k of E experts
      if (tid == 0) {
        list[0] = (int)(blockIdx.y << 8);
        list_n = 1;
      }
      lds_barrier();
      return;
    }
    const int from = padded / 4 * wave / W * 4, to = padded / 4 * (wave + 1) / W * 4;
    if (lane < p.T && from < to) {
      const uint32_t *row = keys + lane * stride;
      atomicAdd(&rank_of[lane], count_before(row, from, to, e));
    }
    lds_barrier();
    if (wave == 0) {
      const int rank = rank_of[lane];
      const bool in = lane < p.T && rank < p.k;
      const uint64_t m = __ballot(in);
      if (in) list[__popcll(m & ((1ull << lane) - 1))] = lane | rank << 8;
      if (lane == 0) list_n = __popcll(m);
    }
    lds_barrier();
  };

  const int r = lane & 15, g = lane >> 4;
  const int f0 = blockIdx.x * (16 * NF), nb = p.H / 32;
  const int rows = p.F - f0 < 16 * NF ? p.F - f0 : 16 * NF;
  const auto [first, last] = steps_of<P>(nb, wave, W);
  const int64_t gate = (int64_t)e * 2 * p.F + f0, up = gate + p.F;
  Rows<2> w;
  set_rows(w, 0, p.up + gate * (p.H / 2), p.up_s + gate * nb, rows, p.H);
  set_rows(w, 1, p.up + up * (p.H / 2), p.up_s + up * nb, rows, p.H);
  Columns<XC> x;
  x.part_bytes = (uint32_t)p.T * p.H * 2;
  x.view = buffer_view(reinterpret_cast<const uint8_t *>(p.xp), NPX * x.part_bytes);
  uint8_t *const mine = lds + wave * Ring::kBytes;
  int n = 0;
  for (int base = 0; base == 0 || base < n; base += 4 * XC) {
    f32x4 acc[2 * NF];
    const auto columns = [&](Columns<XC> &c) {
      if (base == 0) {
        find_tokens();
        n = __builtin_amdgcn_readfirstlane(list_n);
        // several slots can name one expert: the first token's does its work
        if (p.by_slot && (list[0] & 255) != t_first) n = 0;
        if (n == 0) return false;
      }
      set_columns(c, [&](int i) { return base + i < n ? list[base + i] & 255 : -1; }, p.H);
      return true;
    };
    if (!moe_stream<2, NF, XC, NPX, P, SW, SX, ALIGNED>(shared_lds + wave * Ring::kColumns, mine, w, x,
                                                     columns, nb, first, last, acc))
      break;
    keep_sums(mine, acc);
    __syncthreads();
    for (int i = wave; i < NF; i += W) {
      const f32x4 a = sum_of<W>(lds, Ring::kBytes, i), b = sum_of<W>(lds, Ring::kBytes, NF + i);
      bf16x4 part[NPH];
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const float h = a[c] / (1.0f + expf(-a[c])) * b[c];
        __bf16 q[NPH];
        split_bf16<NPH>(h, q);
#pragma unroll
        for (int j = 0; j < NPH; j++) part[j][c] = q[j];
      }
      if (r < 4 * XC && base + r < n && 16 * i < rows) {  // F is a multiple of 32
        const int entry = list[base + r];
        const int64_t slot = (int64_t)(entry & 255) * p.k + (entry >> 8);
#pragma unroll
        for (int j = 0; j < NPH; j++)
          *reinterpret_cast<bf16x4 *>(p.hp + ((int64_t)j * p.T * p.k + slot) * p.F + f0 + 16 * i +
                                      4 * g) = part[j];
      }
    }
    __syncthreads();  // the sums are read before the next loads overwrite them
  }
  if (blockIdx.x == 0) {  // for the down product
    if (tid < n) {
      const int t = list[tid] & 255, slot = t * p.k + (list[tid] >> 8);
      p.slots[blockIdx.y * kMoeTokens + tid] = slot;
      p.chosen_logit[slot] = p.logits[t * p.E + e];
      if (p.by_slot) p.work[slot] = tid == 0 ? e | n << 16 : 0;
    }
    if (!p.by_slot && tid == 0) p.work[e] = e | n << 16;
  }
}

struct DownArgs {
  const __bf16 *hp;
  const int *work, *slots;
  const float *chosen_logit;
  const uint8_t *down, *down_s;
  float *out;
  unsigned *arrived;
  void *y;
  int T, H, F, E, k;
};

// Output rows h0 .. h0+16 NR-1 of one expert for every token that chose it,
// unweighted, by slot.  The workgroup that finds itself the last of its rows
// then adds up the slots of every token, in the order of their ranks and with
// the softmax's weights: the sum has one order, and no fourth kernel is
// needed.  Bound by the weights (as above: 249 MB in 63 us, 4.0 TB/s), for one
// token by latency (8.6 us, 8.9 MB).
template <int TY, int NR, int XC, int W, int P, int SW, int SX, bool ALIGNED>
__global__ __launch_bounds__(W * 64) void moe_down_kernel(DownArgs p) {
  constexpr int NPH = kHParts<TY>;
  typedef MoeRing<1, NR, XC, NPH, P, SW, SX> Ring;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[W * Ring::kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t x_lds[W * Ring::kColumns];
  __shared__ int slots[kMoeTokens], last_one;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  if (tid < kMoeTokens) slots[tid] = p.slots[blockIdx.y * kMoeTokens + tid];
  constexpr int kHold = kMoeTokens * kMoeMaxTopK / (W * 64);
  float chosen_logit[kHold];  // for the last workgroup, which would wait for them
#pragma unroll
  for (int j = 0; j < kHold; j++)
    if (tid + j * W * 64 < p.T * p.k) chosen_logit[j] = p.chosen_logit[tid + j * W * 64];
  const int work = __builtin_amdgcn_readfirstlane(p.work[blockIdx.y]);
  const int e = work & 0xFFFF, n = work >> 16;
  lds_barrier();

  const int h0 = blockIdx.x * (16 * NR), nb = p.F / 32;
  const int rows = p.H - h0 < 16 * NR ? p.H - h0 : 16 * NR;
  const auto [first, last] = steps_of<P>(nb, wave, W);
  const int64_t row0 = (int64_t)e * p.H + h0;
  Rows<1> w;
  set_rows(w, 0, p.down + row0 * (p.F / 2), p.down_s + row0 * nb, rows, p.F);
  Columns<XC> x;
  x.part_bytes = (uint32_t)p.T * p.k * p.F * 2;
  x.view = buffer_view(reinterpret_cast<const uint8_t *>(p.hp), NPH * x.part_bytes);
  const auto out = make_rsrc(p.out, (int64_t)p.T * p.k * p.H * 4);
  uint8_t *const mine = lds + wave * Ring::kBytes;
  for (int base = 0; base < n; base += 4 * XC) {
    f32x4 acc[NR];
    const auto columns = [&](Columns<XC> &c) {
      set_columns(c, [&](int i) { return base + i < n ? slots[base + i] : -1; }, p.F);
      return true;
    };
    moe_stream<1, NR, XC, NPH, P, SW, SX, ALIGNED>(x_lds + wave * Ring::kColumns, mine, w, x, columns,
                                                nb, first, last, acc);
    keep_sums(mine, acc);
    __syncthreads();
    for (int i = wave; i < NR; i += W) {
      const f32x4 v = sum_of<W>(lds, Ring::kBytes, i);
      if (r < 4 * XC && base + r < n && 16 * i < rows)
        __builtin_amdgcn_raw_buffer_store_b128(
            __builtin_bit_cast(u32x4, v), out, (slots[base + r] * p.H + h0 + 16 * i + 4 * g) * 4, 0,
            kCoherent);
    }
    __syncthreads();  // the sums are read before the next loads overwrite them
  }

  // The slots' rows are written and read with the agent-coherent cache policy
  // (written through the XCD's L2, read past its stale lines), every wave
  // waits for its stores before the arrival is counted, and the last one reads
  // only after its count has returned: no write-back of a whole L2 is needed,
  // which release fences here would make (16.2 us of this kernel for one token
  // on 8 of 64 experts of 2048x1024).
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (tid == 0)
    last_one = __hip_atomic_fetch_add(p.arrived + blockIdx.x, 1u, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == gridDim.y - 1;
  __syncthreads();
  if (!last_one) return;
  float *const logit = reinterpret_cast<float *>(lds), *const share = logit + kMoeTokens * kMoeMaxTopK;
#pragma unroll
  for (int j = 0; j < kHold; j++) logit[tid + j * W * 64] = chosen_logit[j];
  __syncthreads();
  if (tid < p.T) {
    const float *l = logit + tid * p.k;
    float sum = 0.0f;
    const float top = l[0];
    for (int i = 0; i < p.k; i++) sum += expf(l[i] - top);
    for (int i = 0; i < p.k; i++) share[tid * p.k + i] = expf(l[i] - top) / sum;
  }
  __syncthreads();
  const int quads = rows / 4;
#pragma unroll 2
  for (int i = tid; i < p.T * quads; i += W * 64) {
    const int t = i / quads, at = h0 + i % quads * 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int q0 = 0; q0 < p.k; q0 += 4) {  // four loads in flight
      f32x4 o[4];
#pragma unroll
      for (int q = 0; q < 4; q++)
        o[q] = __builtin_bit_cast(
            f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       out, q0 + q < p.k ? ((t * p.k + q0 + q) * p.H + at) * 4 : (int)kPastEnd, 0,
                       kCoherent));
#pragma unroll
      for (int q = 0; q < 4; q++)
        if (q0 + q < p.k) v += share[t * p.k + q0 + q] * o[q];
    }
#pragma unroll
    for (int c = 0; c < 4; c++) store_value<TY>(p.y, (int64_t)t * p.H + at + c, v[c]);
  }
}

// Each kernel reads what the one before it writes: the first launch that is
// refused is the last one tried.
template <int TY, bool UP_ALIGNED, bool DOWN_ALIGNED>
hipError_t launch(const MoeArgs &a, const Workspace &w, hipStream_t stream) {
  constexpr int NPX = kXParts<TY>, NPH = kHParts<TY>;
  if (a.T == 1)
    hipLaunchKernelGGL((moe_router_kernel<TY, 1>), dim3(a.E, 1), dim3(256), 0, stream, a.x,
                       a.router, a.bias, w.logits, w.xp, w.arrived, a.T, a.H, a.E);
  else
    hipLaunchKernelGGL((moe_router_kernel<TY, 2>), dim3(a.E, (a.T + 1) / 2), dim3(256), 0, stream,
                       a.x, a.router, a.bias, w.logits, w.xp, w.arrived, a.T, a.H, a.E);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int by_slot = a.T * a.k <= a.E, groups = by_slot ? a.T * a.k : a.E;
  const UpArgs u{TY == MX_BF16 ? static_cast<const __bf16 *>(a.x) : w.xp, w.logits, a.up, a.up_s,
                 w.work, w.slots, w.chosen_logit, w.hp, a.T, a.H, a.F, a.E, a.k, by_slot};
  const DownArgs d{w.hp, w.work, w.slots, w.chosen_logit, a.down, a.down_s, w.out, w.arrived,
                   a.y, a.T, a.H, a.F, a.E, a.k};
  // Wide tiles read the activations less often, narrow ones make more
  // workgroups: the widest that make 512, two for each CU, whose rings fit the
  // CU's LDS twice at least.  The up kernel's keys are not counted: from 54
  // tokens on 128 experts, or 28 on 256, they leave room for one workgroup of
  // the widest bf16 tiles (64 tokens on 8 of 128 experts of 2048x768: 174 us,
  // its weights at the streaming rate 55).
  const auto tiles = [](int rows, int n) { return (rows + 16 * n - 1) / (16 * n); };
  const auto run = [&](auto xc) {
    constexpr int XC = decltype(xc)::value;
    // KiB of a step's activations decide how deep they are kept and how wide a
    // tile fits
    constexpr int kUpX = XC * NPX, kDownX = XC * NPH;
    const auto up = [&](auto nf, auto nw, auto np, auto nsw, auto nsx) {
      constexpr int NF = decltype(nf)::value, W = decltype(nw)::value, P = decltype(np)::value;
      constexpr int SW = decltype(nsw)::value, SX = decltype(nsx)::value;
      hipLaunchKernelGGL((moe_up_kernel<NPX, NPH, NF, XC, W, P, SW, SX, UP_ALIGNED>),
                         dim3(tiles(a.F, NF), groups), dim3(64 * W),
                         std::max((size_t)a.T * key_stride(a.E) * 4,
                                  (size_t)W * MoeRing<2, NF, XC, NPX, P, SW, SX>::kColumns),
                         stream, u);
      e = hipGetLastError();
    };
    const auto down = [&](auto nr, auto nw, auto np, auto nsw, auto nsx) {
      constexpr int NR = decltype(nr)::value, W = decltype(nw)::value, P = decltype(np)::value;
      constexpr int SW = decltype(nsw)::value, SX = decltype(nsx)::value;
      hipLaunchKernelGGL((moe_down_kernel<TY, NR, XC, W, P, SW, SX, DOWN_ALIGNED>),
                         dim3(tiles(a.H, NR), groups), dim3(64 * W), 0, stream, d);
      e = hipGetLastError();
    };
    typedef std::integral_constant<int, 1> I1;
    typedef std::integral_constant<int, 2> I2;
    typedef std::integral_constant<int, 4> I4;
    typedef std::integral_constant<int, (kUpX < 6 ? 3 : 2)> SU;
    typedef std::integral_constant<int, (kUpX == 12 ? 2 : 4)> Wide;
    // Pairs of steps for long rows and many workgroups, where a ring of them
    // leaves wide tiles (32 tokens on 8 experts of 4096x14336 bf16: 192 us
    // against 203; one token on 2 of them 67 against 61).
    bool done = false;
    if constexpr (kUpX <= 4) {
      done = a.H >= 4096 && (int64_t)tiles(a.F, 3) * groups >= 1024;
      if (done) up(std::integral_constant<int, 3>{}, I2{}, I2{}, I2{}, I2{});
    }
    if (done) {
    } else if ((int64_t)tiles(a.F, Wide::value) * groups >= 512) {
      up(Wide{}, I2{}, I1{}, SU{}, SU{});
    } else if ((int64_t)tiles(a.F, 2) * groups >= 512) {
      up(I2{}, I2{}, I1{}, SU{}, SU{});
    } else {
      up(I1{}, std::integral_constant<int, (XC == 1 ? 4 : 2)>{}, I1{}, SU{}, SU{});
    }
    if (e != hipSuccess) return;
    typedef std::integral_constant<int, (XC == 1 ? 4 : 2)> DownWaves;
    typedef std::integral_constant<int, (kDownX == 8 ? 5 : 3)> SDW;
    typedef std::integral_constant<int, (kDownX >= 6 ? 2 : 3)> SDX;
    done = false;
    if constexpr (kDownX <= 8) {
      done = a.F >= 4096 && (int64_t)tiles(a.H, 4) * groups >= 256;
      if (done) down(I4{}, I2{}, I2{}, I2{}, I2{});
    }
    if (done) {
    } else if ((int64_t)tiles(a.H, 4) * groups >= 512) {
      down(I4{}, DownWaves{}, I1{}, SDW{}, SDX{});
    } else {
      down(I2{}, DownWaves{}, I1{}, SDW{}, SDX{});
    }
  };
  // Columns at a time: all of up to four tokens; eight for up to two tokens an
  // expert (an expert that more than eight chose takes its weights again for
  // the next ones, as any beyond 16); 16 otherwise.
  if (a.T <= 4) run(std::integral_constant<int, 1>{});
  else if (a.T * a.k <= 2 * a.E) run(std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 4>{});
  return e;
}

}  // namespace

int64_t moe_workspace_bytes(int64_t T, int64_t H, int64_t F, int64_t E, int64_t k) {
  const int64_t most = moe_tokens_at_once(H, F, E, k);
  return layout(nullptr, MX_F32, T < most ? T : most, H, F, E, k).bytes;
}

hipError_t mxfp4_moe_launch(const MoeArgs &a, hipStream_t stream) {
  const Workspace w = layout(a.workspace, a.type, a.T, a.H, a.F, a.E, a.k);
  const bool up = mx_aligned_scales(a.up_s, a.up_s, a.H);
  const bool down = mx_aligned_scales(a.down_s, a.down_s, a.F);
#define CALL(TY)                                            \
  if (up && down) return launch<TY, true, true>(a, w, stream);     \
  else if (up) return launch<TY, true, false>(a, w, stream);       \
  else if (down) return launch<TY, false, true>(a, w, stream);     \
  else return launch<TY, false, false>(a, w, stream)
  switch (a.type) {
    case MX_F32: CALL(MX_F32);
    case MX_BF16: CALL(MX_BF16);
    default: CALL(MX_F16);
  }
#undef CALL
}

}  // namespace q4k
