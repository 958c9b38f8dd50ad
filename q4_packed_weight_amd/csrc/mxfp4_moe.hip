// mxfp4_moe.hip -- a mixture-of-experts layer of MXFP4 weights for a few
// tokens, as three kernels: the router's logits, the gate and up products
// with the activation between them, and the down product with the sum over
// the chosen experts.
//
// The weights are read once per call and everything else is small, so the
// layer is bound by the weight stream.  e2m1 codes times their block's power
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

// The order of logits as unsigned integers: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t logit_key(float l) {
  if (l != l) return 0u;
  const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Workspace of up to kMoeTokens tokens.
struct Workspace {
  float *logits;        // [T][E]
  int *count;           // [E] tokens of an expert (of a reached one at least)
  int *slots;           // [E][kMoeTokens] their slots: token * k + rank
  int *chosen;          // [T*k] expert of a slot
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
  w.count = reinterpret_cast<int *>(take(E * 4));
  w.slots = reinterpret_cast<int *>(take(E * kMoeTokens * 4));
  w.chosen = reinterpret_cast<int *>(take(T * k * 4));
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
// from zero here.
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

// What a workgroup's waves multiply: V views of NRV tiles of 16 weight rows
// each, and 16 columns of activations in NP bf16 parts.
template <int V, int NRV> struct Rows {
  i32x4 codes[V], scales[V];      // views of the tiles' rows
  const uint8_t *scale_base[V];
  uint32_t code_at[V * NRV];      // this lane's bytes of its row of a load
  uint32_t scale_at[V];           // this lane's row (tile lane / 16, row lane % 16)
};
struct Columns {
  i32x4 view;
  uint32_t at[4], part_bytes;     // this lane's bytes of its row of each load
};

// The rows n0 .. n0+16 NRV-1 (the last one again past `rows`) of a matrix.
template <int V, int NRV>
__device__ __forceinline__ void set_rows(Rows<V, NRV> &w, int v, const uint8_t *codes,
                                         const uint8_t *scales, int rows, int64_t K) {
  const int lane = threadIdx.x & 63;
  const uint32_t bytes = (uint32_t)(K / 2), nb = (uint32_t)(K / 32);
  const auto row = [&](int n) { return (uint32_t)(n < rows ? n : rows - 1); };
  w.codes[v] = buffer_view(codes, (uint32_t)rows * bytes);
  w.scales[v] = buffer_view(scales, (uint32_t)rows * nb);
  w.scale_base[v] = scales;
#pragma unroll
  for (int i = 0; i < NRV; i++)
    w.code_at[v * NRV + i] =
        row(16 * i + tile_row<MX_FP4>(lane)) * bytes + 16 * tile_chunk<MX_FP4>(lane);
  w.scale_at[v] = row(lane) * nb;
}

// 16 columns: `source(i)` is the row of the activations [..][K] of column i,
// negative for none.  A step's 128 positions of a column are 256 bytes, in 16
// chunks of eight values; chunk c is kept at place c ^ (column % 8), so that
// an operand read of eight columns lies on all banks.
template <class F>
__device__ __forceinline__ void set_columns(Columns &x, F source, int64_t K) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int column = 4 * i + (lane >> 4), chunk = (lane & 15) ^ (column & 7);
    const int row = source(column);
    x.at[i] = row < 0 ? kPastEnd : (uint32_t)row * (uint32_t)(2 * K) + 16 * chunk;
  }
}

// The products of steps first .. last-1 of one wave, through a ring of S
// stages of its own in LDS at `ring` (no barrier), the scales of four steps
// behind them.  ALIGNED: rows of whole steps whose scales start at dwords;
// others come through registers, whose wait also waits for what is in flight.
template <int V, int NRV, int NP, int S, bool ALIGNED> struct MoeRing {
  static constexpr int kTiles = V * NRV, kLoads = kTiles + 4 * NP;
  static constexpr int kBytes = (S * kLoads + V) * 1024;
  static_assert(S >= 2 && S <= 4 && NRV <= 4, "");
};
template <int V, int NRV, int NP, int S, bool ALIGNED>
__device__ __forceinline__ void moe_stream(uint8_t *ring, const Rows<V, NRV> &w, const Columns &x,
                                           int nb, int first, int last, f32x4 (&acc)[V * NRV]) {
  typedef MoeRing<V, NRV, NP, S, ALIGNED> R;
  constexpr int kLoads = R::kLoads;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const uint32_t to_ring = lds_address(ring);
  uint8_t *const scales = ring + S * kLoads * 1024;
#pragma unroll
  for (int i = 0; i < R::kTiles; i++) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (first >= last) return;
  const auto issue = [&](int s, int buf) {
    const uint32_t to = to_ring + buf * (kLoads * 1024);
    const bool in_w = ALIGNED || 4 * s + tile_chunk<MX_FP4>(lane) < nb;
#pragma unroll
    for (int i = 0; i < R::kTiles; i++)
      load16_to_lds(w.codes[i / NRV], in_w ? w.code_at[i] + 64u * s : kPastEnd,
                    to + (4 * NP + i) * 1024);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int chunk = (lane & 15) ^ ((4 * i + (lane >> 4)) & 7);
      const bool in_x = ALIGNED || 4 * s + (chunk >> 2) < nb;
#pragma unroll
      for (int q = 0; q < NP; q++)
        load16_to_lds(x.view, in_x ? x.at[i] + q * x.part_bytes + 256u * s : kPastEnd,
                      to + (4 * q + i) * 1024);
    }
  };
  u32x4 held[V];
  const auto load_scales = [&](int s) {
#pragma unroll
    for (int v = 0; v < V; v++)
      if (lane < 16 * NRV) held[v] = load_scales16(w.scale_base[v] + w.scale_at[v], 4 * s, nb);
  };
  const auto issue_scales = [&](int s) {
#pragma unroll
    for (int v = 0; v < V; v++)
      load16_to_lds(w.scales[v], lane < 16 * NRV ? w.scale_at[v] + 4u * s : kPastEnd,
                    to_ring + (S * kLoads + v) * 1024);
  };
  if constexpr (ALIGNED) issue_scales(first);
  else load_scales(first);
#pragma unroll
  for (int d = 0; d < S - 1; d++)
    if (first + d < last) issue(first + d, d);
  int buf = 0;
  uint32_t sc[R::kTiles];
  const auto step = [&](int s, auto jc) {
    constexpr int J = decltype(jc)::value;
    wait_lds();  // what the next loads overwrite is read
    if constexpr (J == 1) {
      if (s + 3 < last) {
        if constexpr (ALIGNED) issue_scales(s + 3);
        else load_scales(s + 3);
      }
    }
    if (s + S - 1 < last) issue(s + S - 1, buf == 0 ? S - 1 : buf - 1);
    // The scales of the steps from s on are older than stage s.
    const int ahead = last - 1 - s;
    if (S > 3 && ahead >= 3) wait_loads<(S > 3 ? 3 : 0) * kLoads>();
    else if (S > 2 && ahead >= 2) wait_loads<(S > 2 ? 2 : 0) * kLoads>();
    else if (ahead >= 1) wait_loads<kLoads>();
    else wait_loads<0>();
    if constexpr (J == 0) {
      if constexpr (!ALIGNED) {
#pragma unroll
        for (int v = 0; v < V; v++)
          if (lane < 16 * NRV) *reinterpret_cast<u32x4 *>(scales + v * 1024 + lane * 16) = held[v];
        wait_lds();
      }
      const uint32_t which = byte_of_two(g);
#pragma unroll
      for (int i = 0; i < R::kTiles; i++)
        sc[i] = byte_of_four(*reinterpret_cast<const u32x4 *>(scales + i / NRV * 1024 +
                                                              i % NRV * 256 + r * 16), which);
    }
    const uint8_t *st = ring + buf * (kLoads * 1024);
    bf16x8 b[NP][4];
#pragma unroll
    for (int q = 0; q < NP; q++)
#pragma unroll
      for (int j = 0; j < 4; j++)
        b[q][j] = *reinterpret_cast<const bf16x8 *>(st + q * 4096 + r * 256 +
                                                    16 * ((4 * g + j) ^ (r & 7)));
#pragma unroll
    for (int i = 0; i < R::kTiles; i++) {
      bf16x8 a[4];
      decode_block(read_operand<MX_FP4>(st + (4 * NP + i) * 1024, operand_at<MX_FP4>(r, g)).v,
                   (sc[i] >> (8 * J)) & 255u, a);
#pragma unroll
      for (int q = 0; q < NP; q++)
#pragma unroll
        for (int j = 0; j < 4; j++)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], b[q][j], acc[i], 0, 0, 0);
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
  int *count, *slots, *chosen;
  float *chosen_logit;
  __bf16 *hp;
  int T, H, F, E, k;
  int by_slot;  // blockIdx.y is a slot, else an expert
};

// Gate and up rows of 16 NF positions of one expert for every token that
// chose it, 16 tokens at a time.  An expert's rank for a token is the number
// of experts before it in the order (logit descending, index ascending), so
// each workgroup finds its tokens by counting, without a sort; ranks below k
// are the chosen ones and give each slot exactly one writer.
template <int NPX, int NPH, int NF, int W, int S, bool ALIGNED>
__global__ __launch_bounds__(W * 64) void moe_up_kernel(UpArgs p) {
  typedef MoeRing<2, NF, NPX, S, ALIGNED> Ring;
  // the logits' keys [T][E] first, the waves' rings later
  constexpr int kBytes = W * Ring::kBytes > kMoeMaxLogits * 4 ? W * Ring::kBytes : kMoeMaxLogits * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kBytes];
  uint32_t *const keys = reinterpret_cast<uint32_t *>(lds);
  __shared__ int rank_of[kMoeTokens];
  __shared__ int list[kMoeTokens];  // token | rank << 8
  __shared__ int found, list_n;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int i = tid; i < p.T * p.E; i += W * 64) keys[i] = logit_key(p.logits[i]);
  __syncthreads();
  int e = blockIdx.y, t_first = -1;
  if (p.by_slot) {
    t_first = blockIdx.y / p.k;
    const int rank = blockIdx.y % p.k;
    for (int q = tid; q < p.E; q += W * 64) {
      const uint32_t *row = keys + t_first * p.E;
      const uint32_t mine = row[q];
      int before = 0;
      for (int i = 0; i < p.E; i++) before += row[i] > mine || (row[i] == mine && i < q);
      if (before == rank) found = q;
    }
    __syncthreads();
    e = __builtin_amdgcn_readfirstlane(found);
  }
  for (int t = wave; t < p.T; t += W) {
    const uint32_t *row = keys + t * p.E;
    const uint32_t mine = row[e];
    int before = 0;
    for (int i = 0; i < p.E; i += 64) {
      const int q = i + lane;
      const bool b = q < p.E && (row[q] > mine || (row[q] == mine && q < e));
      before += __popcll(__ballot(b));
    }
    if (lane == 0) rank_of[t] = before;
  }
  __syncthreads();
  if (wave == 0) {
    const bool in = lane < p.T && rank_of[lane] < p.k;
    const uint64_t m = __ballot(in);
    if (in) list[__popcll(m & ((1ull << lane) - 1))] = lane | rank_of[lane] << 8;
    if (lane == 0) list_n = __popcll(m);
  }
  __syncthreads();
  const int n = __builtin_amdgcn_readfirstlane(list_n);
  // several slots can name one expert: the first token's does its work
  if (p.by_slot && (list[0] & 255) != t_first) return;
  if (blockIdx.x == 0) {
    if (tid == 0) p.count[e] = n;
    if (tid < n) {
      const int t = list[tid] & 255, slot = t * p.k + (list[tid] >> 8);
      p.slots[e * kMoeTokens + tid] = slot;
      p.chosen[slot] = e;
      p.chosen_logit[slot] = p.logits[t * p.E + e];
    }
  }

  const int r = lane & 15, g = lane >> 4;
  const int f0 = blockIdx.x * (16 * NF), nb = p.H / 32, steps = (nb + 3) / 4;
  const int rows = p.F - f0 < 16 * NF ? p.F - f0 : 16 * NF;
  const int first = steps * wave / W, last = steps * (wave + 1) / W;
  const int64_t gate = (int64_t)e * 2 * p.F + f0, up = gate + p.F;
  Rows<2, NF> w;
  set_rows(w, 0, p.up + gate * (p.H / 2), p.up_s + gate * nb, rows, p.H);
  set_rows(w, 1, p.up + up * (p.H / 2), p.up_s + up * nb, rows, p.H);
  Columns x;
  x.part_bytes = (uint32_t)p.T * p.H * 2;
  x.view = buffer_view(reinterpret_cast<const uint8_t *>(p.xp), NPX * x.part_bytes);
  uint8_t *const mine = lds + wave * Ring::kBytes;
  for (int base = 0; base < n; base += 16) {
    if (base) __syncthreads();
    set_columns(x, [&](int i) { return base + i < n ? list[base + i] & 255 : -1; }, p.H);
    f32x4 acc[2 * NF];
    moe_stream<2, NF, NPX, S, ALIGNED>(mine, w, x, nb, first, last, acc);
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
      if (base + r < n && 16 * i < rows) {  // F is a multiple of 32
        const int entry = list[base + r];
        const int64_t slot = (int64_t)(entry & 255) * p.k + (entry >> 8);
#pragma unroll
        for (int j = 0; j < NPH; j++)
          *reinterpret_cast<bf16x4 *>(p.hp + ((int64_t)j * p.T * p.k + slot) * p.F + f0 + 16 * i +
                                      4 * g) = part[j];
      }
    }
  }
}

struct DownArgs {
  const __bf16 *hp;
  const int *count, *slots, *chosen;
  const float *chosen_logit;
  const uint8_t *down, *down_s;
  float *out;
  unsigned *arrived;
  void *y;
  int T, H, F, E, k;
  int by_slot;
};

// Output rows h0 .. h0+16 NR-1 of one expert for every token that chose it,
// unweighted, by slot.  The workgroup that finds itself the last of its rows
// then adds up the slots of every token, in the order of their ranks and with
// the softmax's weights.
template <int TY, int NR, int W, int S, bool ALIGNED>
__global__ __launch_bounds__(W * 64) void moe_down_kernel(DownArgs p) {
  constexpr int NPH = kHParts<TY>;
  typedef MoeRing<1, NR, NPH, S, ALIGNED> Ring;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[W * Ring::kBytes];
  __shared__ int last_one;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int e = __builtin_amdgcn_readfirstlane(p.by_slot ? p.chosen[blockIdx.y] : (int)blockIdx.y);
  const int *slots = p.slots + e * kMoeTokens;
  int n = p.count[e];
  // several slots can name one expert: the first of its list does its work
  if (p.by_slot && slots[0] != (int)blockIdx.y) n = 0;
  n = __builtin_amdgcn_readfirstlane(n);

  const int h0 = blockIdx.x * (16 * NR), nb = p.F / 32, steps = (nb + 3) / 4;
  const int rows = p.H - h0 < 16 * NR ? p.H - h0 : 16 * NR;
  const int first = steps * wave / W, last = steps * (wave + 1) / W;
  const int64_t row0 = (int64_t)e * p.H + h0;
  Rows<1, NR> w;
  set_rows(w, 0, p.down + row0 * (p.F / 2), p.down_s + row0 * nb, rows, p.F);
  Columns x;
  x.part_bytes = (uint32_t)p.T * p.k * p.F * 2;
  x.view = buffer_view(reinterpret_cast<const uint8_t *>(p.hp), NPH * x.part_bytes);
  const auto out = make_rsrc(p.out, (int64_t)p.T * p.k * p.H * 4);
  uint8_t *const mine = lds + wave * Ring::kBytes;
  for (int base = 0; base < n; base += 16) {
    if (base) __syncthreads();
    set_columns(x, [&](int i) { return base + i < n ? slots[base + i] : -1; }, p.F);
    f32x4 acc[NR];
    moe_stream<1, NR, NPH, S, ALIGNED>(mine, w, x, nb, first, last, acc);
    keep_sums(mine, acc);
    __syncthreads();
    for (int i = wave; i < NR; i += W) {
      const f32x4 d = sum_of<W>(lds, Ring::kBytes, i);
      if (base + r < n && 16 * i < rows)
        __builtin_amdgcn_raw_buffer_store_b128(
            __builtin_bit_cast(u32x4, d), out, (slots[base + r] * p.H + h0 + 16 * i + 4 * g) * 4, 0,
            kCoherent);
    }
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
  float *const share = reinterpret_cast<float *>(lds);  // T * k <= 1024
  if (tid < p.T) {
    const float *l = p.chosen_logit + tid * p.k;
    float sum = 0.0f;
    const float top = l[0];
    for (int i = 0; i < p.k; i++) sum += expf(l[i] - top);
    for (int i = 0; i < p.k; i++) share[tid * p.k + i] = expf(l[i] - top) / sum;
  }
  __syncthreads();
  const int quads = rows / 4;
  for (int i = tid; i < p.T * quads; i += W * 64) {
    const int t = i / quads, at = h0 + i % quads * 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int q = 0; q < p.k; q++)
      v += share[t * p.k + q] *
           __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                         out, ((t * p.k + q) * p.H + at) * 4, 0, kCoherent));
#pragma unroll
    for (int c = 0; c < 4; c++) store_value<TY>(p.y, (int64_t)t * p.H + at + c, v[c]);
  }
}

template <int TY, bool UP_ALIGNED, bool DOWN_ALIGNED>
void launch(const MoeArgs &a, const Workspace &w, hipStream_t stream) {
  constexpr int NPX = kXParts<TY>, NPH = kHParts<TY>;
  if (a.T == 1)
    hipLaunchKernelGGL((moe_router_kernel<TY, 1>), dim3(a.E, 1), dim3(256), 0, stream, a.x,
                       a.router, a.bias, w.logits, w.xp, w.arrived, a.T, a.H, a.E);
  else
    hipLaunchKernelGGL((moe_router_kernel<TY, 2>), dim3(a.E, (a.T + 1) / 2), dim3(256), 0, stream,
                       a.x, a.router, a.bias, w.logits, w.xp, w.arrived, a.T, a.H, a.E);
  const int by_slot = a.T * a.k <= a.E, groups = by_slot ? a.T * a.k : a.E;
  const UpArgs u{TY == MX_BF16 ? static_cast<const __bf16 *>(a.x) : w.xp, w.logits, a.up, a.up_s,
                 w.count, w.slots, w.chosen, w.chosen_logit, w.hp, a.T, a.H, a.F, a.E, a.k, by_slot};
  // Wide tiles read the activations less often, narrow ones make more
  // workgroups; two workgroups' rings fit a CU's LDS.
  constexpr int NF = NPX == 3 ? 2 : 4, SU = NPX == 1 ? 3 : 2;
  const auto tiles = [](int rows, int n) { return (rows + 16 * n - 1) / (16 * n); };
  if ((int64_t)tiles(a.F, NF) * groups >= 512)
    hipLaunchKernelGGL((moe_up_kernel<NPX, NPH, NF, 2, SU, UP_ALIGNED>),
                       dim3(tiles(a.F, NF), groups), dim3(128), 0, stream, u);
  else
    hipLaunchKernelGGL((moe_up_kernel<NPX, NPH, 1, 2, (NPX == 1 ? 4 : NPX == 2 ? 3 : 2), UP_ALIGNED>),
                       dim3(tiles(a.F, 1), groups), dim3(128), 0, stream, u);
  const DownArgs d{w.hp, w.count, w.slots, w.chosen, w.chosen_logit, a.down, a.down_s, w.out,
                   w.arrived, a.y, a.T, a.H, a.F, a.E, a.k, by_slot};
  constexpr int SD = NPH == 2 ? 3 : 2;
  if ((int64_t)tiles(a.H, 4) * groups >= 512)
    hipLaunchKernelGGL((moe_down_kernel<TY, 4, 2, SD, DOWN_ALIGNED>), dim3(tiles(a.H, 4), groups),
                       dim3(128), 0, stream, d);
  else
    hipLaunchKernelGGL((moe_down_kernel<TY, 2, 2, SD, DOWN_ALIGNED>), dim3(tiles(a.H, 2), groups),
                       dim3(128), 0, stream, d);
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
  if (up && down) launch<TY, true, true>(a, w, stream);     \
  else if (up) launch<TY, true, false>(a, w, stream);       \
  else if (down) launch<TY, false, true>(a, w, stream);     \
  else launch<TY, false, false>(a, w, stream)
  switch (a.type) {
    case MX_F32: CALL(MX_F32); break;
    case MX_BF16: CALL(MX_BF16); break;
    default: CALL(MX_F16); break;
  }
#undef CALL
  return hipGetLastError();
}

}  // namespace q4k
