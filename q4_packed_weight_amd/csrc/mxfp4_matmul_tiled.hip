// mxfp4_matmul_tiled.hip -- the MX product for many tokens: tiles staged
// through LDS for the scaled matrix instruction.
#include <type_traits>

#include "mx_common.h"
#include "mx_internal.h"

namespace q4k {
namespace {

constexpr int kThreads = 512;
constexpr int kStages = 3;

// One 16-byte piece per lane from a buffer view straight into LDS: lane l's
// lands at lds + 16 l, zeros where the offset is past the view's end.  The
// compiler does not count these loads (they have no destination register);
// wait_loads does.  Nothing else in these kernels uses m0.
__device__ __forceinline__ void load_to_lds(i32x4 view, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(offset), "s"(view)
               : "memory");
}

// Until no more than N of the wave's loads are outstanding.
template <int N> __device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

__device__ __forceinline__ void barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

__device__ __forceinline__ i32x4 buffer_view(const uint8_t *base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32) & 0xFFFF),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

// Scale bytes of 16 consecutive blocks of a row at any alignment; blocks past
// the row's end read as 127.
struct __attribute__((packed)) Packed16 { uint32_t v[4]; };
__device__ __forceinline__ u32x4 load_scales16(const uint8_t *row, int64_t block, int64_t nb) {
  u32x4 r;
  if (block + 16 <= nb) {
    const Packed16 p = *reinterpret_cast<const Packed16 *>(row + block);
    r = u32x4{p.v[0], p.v[1], p.v[2], p.v[3]};
  } else {
    for (int i = 0; i < 4; i++) {
      uint32_t v = 0;
      for (int j = 0; j < 4; j++)
        v |= (uint32_t)(block + 4 * i + j < nb ? row[block + 4 * i + j] : 127) << (8 * j);
      r[i] = v;
    }
  }
  return r;
}

// r[j] holds blocks 4j .. 4j+3 of step j; afterwards dword g holds block g of
// the four steps, one to a byte.
__device__ __forceinline__ u32x4 transpose_bytes(u32x4 r) {
  const uint32_t a = __builtin_amdgcn_perm(r[1], r[0], 0x05010400);  // 0.0 1.0 0.1 1.1
  const uint32_t b = __builtin_amdgcn_perm(r[1], r[0], 0x07030602);  // 0.2 1.2 0.3 1.3
  const uint32_t c = __builtin_amdgcn_perm(r[3], r[2], 0x05010400);
  const uint32_t d = __builtin_amdgcn_perm(r[3], r[2], 0x07030602);
  return u32x4{__builtin_amdgcn_perm(c, a, 0x05040100), __builtin_amdgcn_perm(c, a, 0x07060302),
               __builtin_amdgcn_perm(d, b, 0x05040100), __builtin_amdgcn_perm(d, b, 0x07060302)};
}

// BM tokens x BN weight rows per workgroup of WM x WN waves, each with
// TM x TN tiles of 16x16.
template <int AF, int T, int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(kThreads, 2) void mxfp4_tiled_kernel(
    const uint8_t *a, const uint8_t *as, const uint8_t *w, const uint8_t *ws, void *y, int M,
    int64_t K, int64_t N, int tiles_m, int tiles_n) {
  constexpr int BM = 16 * WM * TM, BN = 16 * WN * TN;
  constexpr int AP = AF == MX_FP4 ? 1 : 2;                // 1 KiB pieces per 16 tokens
  constexpr int kPieces = BM / 16 * AP + BN / 16;         // of a step
  constexpr int kMine = kPieces / 8;
  constexpr int kStage = kPieces * 1024;
  constexpr int kScales = (BM + BN) * 16;
  static_assert(kPieces % 8 == 0 && BM + BN <= kThreads, "");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kStages * kStage + 2 * kScales];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;

  // Workgroups go to the 8 XCDs in turn: each XCD takes a run of tiles, eight
  // token tiles deep, so that its L2 serves the tiles that share operands.
  const int tiles = tiles_m * tiles_n;
  int id = blockIdx.x;
  {
    const int per = tiles / 8, more = tiles % 8, x = id & 7;
    id = (id >> 3) + x * per + (x < more ? x : more);
  }
  constexpr int kDeep = 8;
  const int group = id / (kDeep * tiles_n), in = id % (kDeep * tiles_n);
  const int deep = tiles_m - group * kDeep < kDeep ? tiles_m - group * kDeep : kDeep;
  const int bm = group * kDeep + in % deep, bn = in / deep;
  const int m0 = bm * BM;
  const int64_t n0 = (int64_t)bn * BN;
  const int rows_m = M - m0 < BM ? M - m0 : BM, rows_n = N - n0 < BN ? (int)(N - n0) : BN;

  const int64_t nb = K / 32;
  const int steps = (int)((nb + 3) / 4);
  const uint32_t a_bytes = (uint32_t)(AF == MX_FP4 ? K / 2 : K), w_bytes = (uint32_t)(K / 2);
  const i32x4 a_view = buffer_view(a + (int64_t)m0 * a_bytes, rows_m * a_bytes);
  const i32x4 w_view = buffer_view(w + n0 * w_bytes, rows_n * w_bytes);

  // A piece is 1 KiB: 8 rows x 128 bytes (e4m3) or 16 rows x 64 (e2m1), with
  // neighbouring lanes on neighbouring bytes of a row.  The 16-byte chunks of
  // a row are stored in an order that changes with the row (chunk c at place
  // c ^ spread), so that the 16 rows a fragment read takes lie on all banks.
  // Weight rows go to the tiles in pairs: the lane that ends with rows
  // 4g .. 4g+3 of both tiles of a pair has eight consecutive outputs.
  uint32_t offset[kMine];
  int chunk[kMine];
#pragma unroll
  for (int i = 0; i < kMine; i++) {
    const int p = i * 8 + wave;
    if (p < BM / 16 * AP) {
      const int row = AP == 2 ? lane >> 3 : lane >> 2;
      const int m = p * (16 / AP) + row;
      chunk[i] = AP == 2 ? (lane & 7) ^ row : (lane & 3) ^ ((row >> 1) & 3);
      offset[i] = (uint32_t)(m < rows_m ? m : rows_m - 1) * a_bytes + 16 * chunk[i];
    } else {
      const int t = p - BM / 16 * AP, row = lane >> 2;
      const int n = (t >> 1) * 32 + (row >> 2) * 8 + (t & 1) * 4 + (row & 3);
      chunk[i] = (lane & 3) ^ ((row >> 1) & 3);
      offset[i] = (uint32_t)(n < rows_n ? n : rows_n - 1) * w_bytes + 16 * chunk[i];
    }
  }
  // where a lane finds the chunks of its row in a 16-row tile
  const int at_w = r * 64 + 16 * (g ^ ((r >> 1) & 3));
  const int at_a = AP == 2 ? r * 128 + 16 * (g ^ (r & 7)) : at_w;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void *)lds;
  const int whole = (int)(nb / 4);  // steps of four blocks
  const auto issue = [&](int s, int buf) {
    const int blocks = (int)(nb - 4 * (int64_t)s);
#pragma unroll
    for (int i = 0; i < kMine; i++) {
      const int p = i * 8 + wave;
      const bool is_a = p < BM / 16 * AP;
      uint32_t o = offset[i] + (uint32_t)s * (is_a ? 64 * AP : 64);
      if (s >= whole) {  // the row's last blocks: zeros after them
        const int block = is_a && AP == 2 ? chunk[i] >> 1 : chunk[i];
        if (block >= blocks) o = 0x7FFFFFF0u;
      }
      load_to_lds(is_a ? a_view : w_view, o, lds0 + buf * kStage + p * 1024);
    }
  };

  // Scales of four steps at a time, one row (token or weight) per thread.
  const bool has_row = tid < BM + BN;
  const uint8_t *scale_row;
  if (tid < BM) scale_row = as + (int64_t)(m0 + (tid < rows_m ? tid : rows_m - 1)) * nb;
  else scale_row = ws + (n0 + (tid - BM < rows_n ? tid - BM : rows_n - 1)) * nb;
  uint8_t *const scales = lds + kStages * kStage;

  const int wm = wave % WM, wn = wave / WM;
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; i++)
#pragma unroll
    for (int j = 0; j < TN; j++) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  u32x4 next = {0, 0, 0, 0};
  if (has_row) {
    next = load_scales16(scale_row, 0, nb);
    *reinterpret_cast<u32x4 *>(scales + tid * 16) = transpose_bytes(next);
  }
  issue(0, 0);
  if (steps > 1) {
    issue(1, 1);
    wait_loads<kMine>();
  } else {
    wait_loads<0>();
  }
  barrier();

  // Each SIMD holds one wave of the first four and one of the others, and the
  // second four run one barrier behind: while one wave of a SIMD multiplies a
  // step, the other fetches its operands from LDS and sends the loads of two
  // steps on.  A stage is overwritten after both halves have fetched from it,
  // and read after the barrier that follows every wave's wait for it.
  const bool behind = wave >= 4;
  if (behind) barrier();
  int buf = 0;
  int sa[TM], sw[TN];
  const auto step = [&](int s, auto jc) {
    constexpr int J = decltype(jc)::value;
    if constexpr (J == 3) {  // read two barriers on, by both halves
      if (has_row && s + 1 < steps)
        *reinterpret_cast<u32x4 *>(scales + (((s >> 2) + 1) & 1) * kScales + tid * 16) =
            transpose_bytes(next);
    }
    const uint8_t *st = lds + buf * kStage;
    i32x8 ta[TM];
    i32x4 tw[TN];
#pragma unroll
    for (int i = 0; i < TM; i++) {
      const uint8_t *p = st + (wm * TM + i) * AP * 1024;
      const i32x4 lo = *reinterpret_cast<const i32x4 *>(p + at_a);
      i32x4 hi = {0, 0, 0, 0};
      if constexpr (AP == 2) hi = *reinterpret_cast<const i32x4 *>(p + (at_a ^ 64));
      ta[i] = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
#pragma unroll
    for (int j = 0; j < TN; j++)
      tw[j] = *reinterpret_cast<const i32x4 *>(st + (BM / 16 * AP + wn * TN + j) * 1024 + at_w);
    if constexpr (J == 0) {
      const uint8_t *sc = scales + ((s >> 2) & 1) * kScales;
#pragma unroll
      for (int i = 0; i < TM; i++)
        sa[i] = *reinterpret_cast<const int *>(sc + ((wm * TM + i) * 16 + r) * 16 + 4 * g);
#pragma unroll
      for (int j = 0; j < TN; j++) {
        const int t = wn * TN + j;
        const int n = (t >> 1) * 32 + (r >> 2) * 8 + (t & 1) * 4 + (r & 3);
        sw[j] = *reinterpret_cast<const int *>(sc + (BM + n) * 16 + 4 * g);
      }
      if (has_row && s + 4 < steps) next = load_scales16(scale_row, 4 * (int64_t)(s + 4), nb);
    }
    if (s + 2 < steps) {
      issue(s + 2, buf == 0 ? 2 : buf - 1);
      wait_loads<kMine>();
    } else {
      wait_loads<0>();
    }
    barrier();
    __builtin_amdgcn_sched_barrier(0);
    const auto multiply = [&](int i, int j) {
      const i32x8 v = {tw[j][0], tw[j][1], tw[j][2], tw[j][3], 0, 0, 0, 0};
      acc[i][j] = mfma_mx<MX_FP4, AF, T == MX_F32, J>(v, ta[i], acc[i][j], sw[j], sa[i]);
    };
    if constexpr (T == MX_F32 && AF == MX_FP8) {  // tokens outside: each is split in two once
#pragma unroll
      for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) multiply(i, j);
    } else {
#pragma unroll
      for (int j = 0; j < TN; j++)
#pragma unroll
        for (int i = 0; i < TM; i++) multiply(i, j);
    }
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    __builtin_amdgcn_sched_barrier(0);
    buf = buf == 2 ? 0 : buf + 1;
  };
  for (int s = 0; s < steps; s += 4) {
    step(s, std::integral_constant<int, 0>{});
    if (s + 1 < steps) step(s + 1, std::integral_constant<int, 1>{});
    if (s + 2 < steps) step(s + 2, std::integral_constant<int, 2>{});
    if (s + 3 < steps) step(s + 3, std::integral_constant<int, 3>{});
  }
  if (!behind) barrier();

  typedef typename MxStore<T>::type Out;
  Out *const yo = static_cast<Out *>(y);
  const bool wide = N % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
#pragma unroll
  for (int i = 0; i < TM; i++) {
    const int m = (wm * TM + i) * 16 + r;
    if (m >= rows_m) continue;
#pragma unroll
    for (int j = 0; j < TN; j += 2) {
      const int n = (wn * TN + j) * 16 + 8 * g;
      const int64_t at = (int64_t)(m0 + m) * N + n0 + n;
      float f[8];
#pragma unroll
      for (int q = 0; q < 4; q++) {
        f[q] = acc[i][j][q];
        f[4 + q] = acc[i][j + 1][q];
      }
      if (wide && n + 8 <= rows_n) {
        store_raw8<T>(yo + at, 0, f32_to_raw8<T>(f));
      } else {
#pragma unroll
        for (int q = 0; q < 8; q++)
          if (n + q < rows_n) yo[at + q] = (Out)f[q];
      }
    }
  }
}

template <int AF, int T, int WM, int WN, int TM, int TN>
void launch(const uint8_t *a, const uint8_t *as, const uint8_t *w, const uint8_t *ws, int M,
            int64_t K, int64_t N, void *Y, hipStream_t stream) {
  const int tm = (M + 16 * WM * TM - 1) / (16 * WM * TM);
  const int tn = (int)((N + 16 * WN * TN - 1) / (16 * WN * TN));
  hipLaunchKernelGGL((mxfp4_tiled_kernel<AF, T, WM, WN, TM, TN>), dim3(tm * tn), dim3(kThreads), 0,
                     stream, a, as, w, ws, Y, M, K, N, tm, tn);
}

}  // namespace

hipError_t mxfp4_matmul_tiled_launch(const uint8_t *a, const uint8_t *as, int a_format,
                                     const uint8_t *w, const uint8_t *ws, int64_t M, int64_t K,
                                     int64_t N, void *Y, int type, hipStream_t stream) {
#define CALL(AF)                                                                                  \
  switch (type) {                                                                                 \
    case MX_F32: launch<AF, MX_F32, 4, 2, 4, 8>(a, as, w, ws, (int)M, K, N, Y, stream); break;    \
    case MX_BF16: launch<AF, MX_BF16, 4, 2, 4, 8>(a, as, w, ws, (int)M, K, N, Y, stream); break;  \
    default: launch<AF, MX_F16, 4, 2, 4, 8>(a, as, w, ws, (int)M, K, N, Y, stream); break;        \
  }
  if (a_format == MX_FP4) { CALL(MX_FP4) } else { CALL(MX_FP8) }
#undef CALL
  return hipGetLastError();
}

}  // namespace q4k
