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
#include <type_traits>

#include "mx_common.h"
#include "mx_internal.h"

namespace q4k {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kUpWaves = 4;

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

// Workspace of up to kMoeTokens tokens, in order: logits, chosen experts and
// their logits by (token, rank), x in bf16 parts, h in bf16 parts.
struct Workspace {
  float *logits;       // [T][E]
  int *chosen;         // [T][k]
  float *chosen_logit; // [T][k]
  __bf16 *xp;          // [NPX][T][H], none for bf16 x
  __bf16 *hp;          // [NPH][T*k][F]
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
  w.logits = reinterpret_cast<float *>(p + o);
  o += align256(T * E * 4);
  w.chosen = reinterpret_cast<int *>(p + o);
  o += align256(T * k * 4);
  w.chosen_logit = reinterpret_cast<float *>(p + o);
  o += align256(T * k * 4);
  w.xp = reinterpret_cast<__bf16 *>(p + o);
  o += align256(px * T * H * 2);
  w.hp = reinterpret_cast<__bf16 *>(p + o);
  o += align256(ph * T * k * F * 2);
  w.bytes = o;
  return w;
}

// logits[t, e] for TT tokens per workgroup and one expert; the workgroups
// also share out the splitting of x.
template <int TY, int TT>
__global__ __launch_bounds__(256) void moe_router_kernel(const void *x, const void *router,
                                                         const float *bias, float *logits,
                                                         __bf16 *xp, int T, int H, int E) {
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

struct UpArgs {
  const __bf16 *xp;
  const float *logits;
  const uint8_t *up, *up_s;
  int *chosen;
  float *chosen_logit;
  __bf16 *hp;
  int T, H, F, E, k;
  int by_slot;  // blockIdx.y is a (token, rank), else an expert
};

// Gate and up rows f0 .. f0+15 of one expert for every token that chose it.
// An expert's rank for a token is the number of experts before it in the
// order (logit descending, index ascending), so each workgroup finds its
// tokens by counting, without a sort; ranks below k are the chosen ones and
// give each (token, rank) exactly one writer.
template <int NPX, int NPH, int NT>
__global__ __launch_bounds__(kUpWaves * 64) void moe_up_kernel(UpArgs p) {
  // the logits' keys [T][E] first, the waves' partial tiles [kUpWaves][NT][2][64] later
  extern __shared__ f32x4 lds[];
  uint32_t *keys = reinterpret_cast<uint32_t *>(lds);
  auto red = reinterpret_cast<f32x4(*)[NT][2][64]>(lds);
  __shared__ int rank_of[kMoeTokens];
  __shared__ int list[kMoeTokens];  // token | rank << 8
  __shared__ int found, list_n;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < p.T * p.E; i += kUpWaves * 64) keys[i] = logit_key(p.logits[i]);
  __syncthreads();
  int e = blockIdx.y, t_first = -1;
  if (p.by_slot) {
    t_first = blockIdx.y / p.k;
    const int rank = blockIdx.y % p.k;
    if (tid < p.E) {
      const uint32_t *row = keys + t_first * p.E;
      const uint32_t mine = row[tid];
      int before = 0;
      for (int i = 0; i < p.E; i++) before += row[i] > mine || (row[i] == mine && i < tid);
      if (before == rank) found = tid;
    }
    __syncthreads();
    e = found;
  }
  for (int t = wave; t < p.T; t += kUpWaves) {
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
  const int n = list_n;
  if (n == 0) return;
  // several slots can name one expert: the first token's does its work
  if (p.by_slot && (list[0] & 255) != t_first) return;
  if (blockIdx.x == 0 && tid < n) {
    const int t = list[tid] & 255, rank = list[tid] >> 8;
    p.chosen[t * p.k + rank] = e;
    p.chosen_logit[t * p.k + rank] = p.logits[t * p.E + e];
  }

  const int r = lane & 15, g = lane >> 4;
  const int f0 = blockIdx.x * 16, nb = p.H / 32, steps = (nb + 3) / 4;
  const int nt = (n + 15) / 16;
  const int64_t gate = (int64_t)e * 2 * p.F + f0 + r, up = gate + p.F;
  const uint8_t *gw = p.up + gate * (p.H / 2), *uw = p.up + up * (p.H / 2);
  const uint8_t *gs = p.up_s + gate * nb, *us = p.up_s + up * nb;
  const __bf16 *xrow[NT];
#pragma unroll
  for (int t = 0; t < NT; t++) {
    const int i = 16 * t + r < n ? 16 * t + r : n - 1;
    xrow[t] = p.xp + (int64_t)(list[i] & 255) * p.H;
  }
  f32x4 ag[NT], au[NT];
#pragma unroll
  for (int t = 0; t < NT; t++) ag[t] = au[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = wave; s < steps; s += kUpWaves) {
    const int kb = 4 * s + g;
    const bool in = kb < nb;
    i32x4 gc = {0, 0, 0, 0}, uc = {0, 0, 0, 0};
    uint32_t gsc = 127, usc = 127;
    if (in) {
      gc = *reinterpret_cast<const i32x4 *>(gw + 16 * kb);
      uc = *reinterpret_cast<const i32x4 *>(uw + 16 * kb);
      gsc = gs[kb];
      usc = us[kb];
    }
    bf16x8 ga[4], ua[4];
    decode_block(gc, gsc, ga);
    decode_block(uc, usc, ua);
#pragma unroll
    for (int t = 0; t < NT; t++) {
      if (t < nt) {
#pragma unroll
        for (int q = 0; q < NPX; q++) {
          const __bf16 *x = xrow[t] + (int64_t)q * p.T * p.H + 32 * kb;
#pragma unroll
          for (int j = 0; j < 4; j++) {
            bf16x8 b = {};
            if (in) b = *reinterpret_cast<const bf16x8 *>(x + 8 * j);
            ag[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ga[j], b, ag[t], 0, 0, 0);
            au[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ua[j], b, au[t], 0, 0, 0);
          }
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; t++) {
    red[wave][t][0][lane] = ag[t];
    red[wave][t][1][lane] = au[t];
  }
  __syncthreads();
  for (int t = wave; t < nt; t += kUpWaves) {
    f32x4 a = red[0][t][0][lane], b = red[0][t][1][lane];
#pragma unroll
    for (int i = 1; i < kUpWaves; i++) {
      a += red[i][t][0][lane];
      b += red[i][t][1][lane];
    }
    bf16x4 part[NPH];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float h = a[i] / (1.0f + expf(-a[i])) * b[i];
      __bf16 q[NPH];
      split_bf16<NPH>(h, q);
#pragma unroll
      for (int j = 0; j < NPH; j++) part[j][i] = q[j];
    }
    if (16 * t + r < n) {
      const int entry = list[16 * t + r];
      const int64_t slot = (int64_t)(entry & 255) * p.k + (entry >> 8);
#pragma unroll
      for (int j = 0; j < NPH; j++)
        *reinterpret_cast<bf16x4 *>(p.hp + ((int64_t)j * p.T * p.k + slot) * p.F + f0 + 4 * g) =
            part[j];
    }
  }
}

struct DownArgs {
  const __bf16 *hp;
  const int *chosen;
  const float *chosen_logit;
  const uint8_t *down, *down_s;
  void *y;
  int T, H, F, E, k;
};

// Output rows h0 .. h0+15 for every token.  The reached experts' 128-position
// steps form one sequence, cut evenly between the waves; a wave that leaves an
// expert adds its tile, weighted, to its own fp32 rows in LDS, and the waves'
// rows are added in order at the end.
template <int TY, int NT, int W>
__global__ __launch_bounds__(W * 64) void moe_down_kernel(DownArgs p) {
  constexpr int NPH = kHParts<TY>;
  constexpr int kMost = NT * 16 * kMoeMaxTopK;  // (token, rank) pairs
  __shared__ int expert_of[kMost];
  __shared__ float share[kMost];
  __shared__ short list[kMost];            // pairs by expert
  __shared__ int start[kMoeMaxExperts + 1];  // of the reached experts' pairs
  __shared__ short reached[kMoeMaxExperts];
  __shared__ int n_reached;
  __shared__ int count[kMoeMaxExperts];
  __shared__ f32x4 out[W][NT * 16][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int pairs = p.T * p.k;
  for (int i = tid; i < pairs; i += W * 64) expert_of[i] = p.chosen[i];
  if (tid < p.T) {
    const float *l = p.chosen_logit + tid * p.k;
    float sum = 0.0f;
    const float top = l[0];
    for (int i = 0; i < p.k; i++) sum += expf(l[i] - top);
    for (int i = 0; i < p.k; i++) share[tid * p.k + i] = expf(l[i] - top) / sum;
  }
#pragma unroll
  for (int i = 0; i < NT; i++) out[wave][i * 16 + (lane >> 2)][lane & 3] = f32x4{0, 0, 0, 0};
  __syncthreads();
  for (int e = tid; e < p.E; e += W * 64) {
    int c = 0;
    for (int i = 0; i < pairs; i++) c += expert_of[i] == e;
    count[e] = c;
  }
  __syncthreads();
  if (tid == 0) {
    int at = 0, m = 0;
    for (int e = 0; e < p.E; e++)
      if (count[e] > 0) {
        start[m] = at;
        reached[m++] = (short)e;
        at += count[e];
      }
    start[m] = at;
    n_reached = m;
  }
  __syncthreads();
  for (int j = tid; j < n_reached; j += W * 64) {
    int at = start[j];
    for (int i = 0; i < pairs; i++)
      if (expert_of[i] == reached[j]) list[at++] = (short)i;
  }
  __syncthreads();

  const int r = lane & 15, g = lane >> 4;
  const int h0 = blockIdx.x * 16, nb = p.F / 32, steps = (nb + 3) / 4;
  const int64_t total = (int64_t)n_reached * steps;
  int64_t at = total * wave / W;
  const int64_t last = total * (wave + 1) / W;
  while (at < last) {
    const int j = (int)(at / steps);
    int s = (int)(at % steps);
    const int s_end = last - (int64_t)j * steps < steps ? (int)(last - (int64_t)j * steps) : steps;
    at += s_end - s;
    const int first = start[j], n = start[j + 1] - first, nt = (n + 15) / 16;
    const int64_t row = (int64_t)reached[j] * p.H + h0 + r;
    const uint8_t *w = p.down + row * (p.F / 2), *ws = p.down_s + row * nb;
    const __bf16 *hrow[NT];
#pragma unroll
    for (int t = 0; t < NT; t++)
      hrow[t] = p.hp + (int64_t)list[first + (16 * t + r < n ? 16 * t + r : n - 1)] * p.F;
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (; s < s_end; s++) {
      const int kb = 4 * s + g;
      const bool in = kb < nb;
      i32x4 c = {0, 0, 0, 0};
      uint32_t sc = 127;
      if (in) {
        c = *reinterpret_cast<const i32x4 *>(w + 16 * kb);
        sc = ws[kb];
      }
      bf16x8 a[4];
      decode_block(c, sc, a);
#pragma unroll
      for (int t = 0; t < NT; t++) {
        if (t < nt) {
#pragma unroll
          for (int q = 0; q < NPH; q++) {
            const __bf16 *h = hrow[t] + (int64_t)q * pairs * p.F + 32 * kb;
#pragma unroll
            for (int i = 0; i < 4; i++) {
              bf16x8 b = {};
              if (in) b = *reinterpret_cast<const bf16x8 *>(h + 8 * i);
              acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b, acc[t], 0, 0, 0);
            }
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; t++) {
      if (16 * t + r < n) {
        const int pair = list[first + 16 * t + r];
        out[wave][pair / p.k][g] += share[pair] * acc[t];
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < p.T * 16; i += W * 64) {
    const int t = i >> 4, row = i & 15;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < W; q++) v += out[q][t][row >> 2][row & 3];
    store_value<TY>(p.y, (int64_t)t * p.H + h0 + row, v);
  }
}

template <int TY, int NT>
void launch(const MoeArgs &a, const Workspace &w, hipStream_t stream) {
  constexpr int NPX = kXParts<TY>, NPH = kHParts<TY>;
  constexpr int W = NT == 1 ? 16 : 8;
  if (a.T == 1)
    hipLaunchKernelGGL((moe_router_kernel<TY, 1>), dim3(a.E, 1), dim3(256), 0, stream, a.x,
                       a.router, a.bias, w.logits, w.xp, a.T, a.H, a.E);
  else
    hipLaunchKernelGGL((moe_router_kernel<TY, 8>), dim3(a.E, (a.T + 7) / 8), dim3(256), 0, stream,
                       a.x, a.router, a.bias, w.logits, w.xp, a.T, a.H, a.E);
  UpArgs u{TY == MX_BF16 ? static_cast<const __bf16 *>(a.x) : w.xp, w.logits, a.up, a.up_s,
           w.chosen, w.chosen_logit, w.hp, a.T, a.H, a.F, a.E, a.k, a.T * a.k <= a.E};
  const size_t keys = (size_t)a.T * a.E * 4, red = sizeof(f32x4) * kUpWaves * NT * 2 * 64;
  const size_t lds = keys > red ? keys : red;
  hipLaunchKernelGGL((moe_up_kernel<NPX, NPH, NT>),
                     dim3(a.F / 16, u.by_slot ? a.T * a.k : a.E), dim3(kUpWaves * 64),
                     lds, stream, u);
  DownArgs d{w.hp, w.chosen, w.chosen_logit, a.down, a.down_s, a.y, a.T, a.H, a.F, a.E, a.k};
  hipLaunchKernelGGL((moe_down_kernel<TY, NT, W>), dim3(a.H / 16), dim3(W * 64), 0, stream, d);
}

}  // namespace

int64_t moe_workspace_bytes(int64_t T, int64_t H, int64_t F, int64_t E, int64_t k) {
  const int64_t most = moe_tokens_at_once(E);
  return layout(nullptr, MX_F32, T < most ? T : most, H, F, E, k).bytes;
}

hipError_t mxfp4_moe_launch(const MoeArgs &a, hipStream_t stream) {
  const Workspace w = layout(a.workspace, a.type, a.T, a.H, a.F, a.E, a.k);
#define CALL(TY)                       \
  if (a.T <= 16) launch<TY, 1>(a, w, stream); \
  else launch<TY, 4>(a, w, stream)
  switch (a.type) {
    case MX_F32: CALL(MX_F32); break;
    case MX_BF16: CALL(MX_BF16); break;
    default: CALL(MX_F16); break;
  }
#undef CALL
  return hipGetLastError();
}

}  // namespace q4k
