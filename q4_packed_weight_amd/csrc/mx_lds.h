// mx_lds.h -- MX operands through LDS: loads that go there straight from
// memory, the order they are kept in, and the reads of matrix operands.
#pragma once

#include "mx_common.h"

namespace q4k {

// One piece per lane from a buffer view straight into LDS: lane l's lands at
// lds + 16 l, zeros where the offset is past the view's end.  ONCE: with the
// non-temporal hint.  The compiler does not count these loads (they have no
// destination register); wait_loads does.  Nothing else in the kernels that
// include this uses m0.
template <bool ONCE = false>
__device__ __forceinline__ void load16_to_lds(i32x4 view, uint32_t offset, uint32_t lds) {
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
                 :
                 : "s"(lds), "v"(offset), "s"(view)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(offset), "s"(view)
                 : "memory");
}

// Until no more than N of the wave's loads are outstanding.
template <int N> __device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "the counter has six bits");
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// Until the wave's LDS reads and writes are done.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

__device__ __forceinline__ i32x4 buffer_view(const uint8_t *base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32) & 0xFFFF),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

constexpr uint32_t kPastEnd = 0x7FFFFFF0u;  // of every view: reads as zeros

__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

// A 16-row tile's 128 positions lie in LDS as 2 KiB (MX_FP8, two loads of a
// wave, 8 rows x 128 bytes each) or 1 KiB (MX_FP4, one load of 16 rows x 64
// bytes), neighbouring lanes on neighbouring bytes of a row: loads whose
// neighbouring lanes lie in different rows ran 1.5 times slower (4096x4096 by
// 16384x4096: 378 against 255 us for the loads alone).  The 16-byte chunks of
// a row are stored in an order that changes with the row, so that the eight
// rows an operand read takes at a time lie on all banks.
template <int F> constexpr int kTileLoads = F == MX_FP8 ? 2 : 1;
template <int F> __device__ __forceinline__ int tile_row(int lane) {  // within its load
  return F == MX_FP8 ? lane >> 3 : lane >> 2;
}
template <int F> __device__ __forceinline__ int tile_chunk(int lane) {
  const int row = tile_row<F>(lane);
  return F == MX_FP8 ? (lane & 7) ^ row : (lane & 3) ^ ((row >> 1) & 3);
}
// The block of four that a chunk belongs to.
template <int F> __device__ __forceinline__ int chunk_block(int chunk) {
  return F == MX_FP8 ? chunk >> 1 : chunk;
}
// Operand of the tile at p: lane (r, g) as mfma_scaled takes it.
template <int F> __device__ __forceinline__ int operand_at(int r, int g) {
  return F == MX_FP8 ? r * 128 + 16 * (g ^ (r & 7)) : r * 64 + 16 * (g ^ ((r >> 1) & 3));
}
template <int F> struct Operand;
template <> struct Operand<MX_FP8> { i32x8 v; };
template <> struct Operand<MX_FP4> { i32x4 v; };
template <int F> __device__ __forceinline__ Operand<F> read_operand(const uint8_t *p, int at) {
  const i32x4 lo = *reinterpret_cast<const i32x4 *>(p + at);
  if constexpr (F == MX_FP8) {
    const i32x4 hi = *reinterpret_cast<const i32x4 *>(p + (at ^ 64));
    return {i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}};
  } else {
    return {lo};
  }
}
__device__ __forceinline__ i32x8 eight(Operand<MX_FP8> o) { return o.v; }
__device__ __forceinline__ i32x8 eight(Operand<MX_FP4> o) {
  return i32x8{o.v[0], o.v[1], o.v[2], o.v[3], 0, 0, 0, 0};
}

// Weight rows go to tiles in pairs: row r of tile t of a pair-wise interleaved
// run, so that the lane that ends with rows 4g .. 4g+3 of both tiles of a pair
// has eight consecutive outputs.
__device__ __forceinline__ int paired_row(int tile, int r) {
  return (tile >> 1) * 32 + (r >> 2) * 8 + (tile & 1) * 4 + (r & 3);
}

// Scale bytes of 16 consecutive blocks of a row at any alignment; blocks past
// the row's end read as 127.
struct __attribute__((packed)) Packed16 { uint32_t v[4]; };
__device__ __forceinline__ u32x4 load_scales16(const uint8_t *row, int64_t block, int64_t nb) {
  constexpr uint32_t kOnes = 0x7F7F7F7Fu;
  u32x4 r = {kOnes, kOnes, kOnes, kOnes};
  const auto load = [&](int64_t at) {
    const Packed16 p = *reinterpret_cast<const Packed16 *>(row + at);
    return u32x4{p.v[0], p.v[1], p.v[2], p.v[3]};
  };
  if (block + 16 <= nb) {
    r = load(block);
  } else if (block < nb && nb >= 16) {
    // the row's last 16, moved down: byte by byte the tail is 16 loads in turn
    // (8 tokens, 4096 x 1056: 5.1 us, so 3.7)
    const int past = (int)(block + 16 - nb);
    r = load(nb - 16);
    if (past & 8) r = u32x4{r[2], r[3], kOnes, kOnes};
    if (past & 4) r = u32x4{r[1], r[2], r[3], kOnes};
    const uint32_t w[5] = {r[0], r[1], r[2], r[3], kOnes};
#pragma unroll
    for (int i = 0; i < 4; i++) r[i] = __builtin_amdgcn_alignbyte(w[i + 1], w[i], past & 3);
  } else if (block < nb) {
    for (int i = 0; i < 4; i++) {
      uint32_t v = 0;
      for (int j = 0; j < 4; j++)
        v |= (uint32_t)(block + 4 * i + j < nb ? row[block + 4 * i + j] : 127) << (8 * j);
      r[i] = v;
    }
  }
  return r;
}

// Byte g of each of four dwords, in order: `which` is byte_of_two(g).
__device__ __forceinline__ uint32_t byte_of_two(int g) { return (uint32_t)(g | (4 + g) << 8); }
__device__ __forceinline__ uint32_t byte_of_four(u32x4 v, uint32_t which) {
  const uint32_t lo = __builtin_amdgcn_perm(v[1], v[0], which);
  const uint32_t hi = __builtin_amdgcn_perm(v[3], v[2], which);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100);
}

// Dword g of the result is byte g of each of the four, in order.
__device__ __forceinline__ u32x4 transpose_bytes(u32x4 r) {
  const uint32_t a = __builtin_amdgcn_perm(r[1], r[0], 0x05010400);  // 0.0 1.0 0.1 1.1
  const uint32_t b = __builtin_amdgcn_perm(r[1], r[0], 0x07030602);  // 0.2 1.2 0.3 1.3
  const uint32_t c = __builtin_amdgcn_perm(r[3], r[2], 0x05010400);
  const uint32_t d = __builtin_amdgcn_perm(r[3], r[2], 0x07030602);
  return u32x4{__builtin_amdgcn_perm(c, a, 0x05040100), __builtin_amdgcn_perm(c, a, 0x07060302),
               __builtin_amdgcn_perm(d, b, 0x05040100), __builtin_amdgcn_perm(d, b, 0x07060302)};
}

// Eight consecutive outputs of a row of N, of which `left` exist.
template <int T>
__device__ __forceinline__ void store_row8(void *y, int64_t at, const float (&f)[8], int left,
                                           bool wide) {
  typedef typename MxStore<T>::type Out;
  Out *const p = static_cast<Out *>(y) + at;
  if (wide && left >= 8) {
    store_raw8<T>(p, 0, f32_to_raw8<T>(f));
  } else {
#pragma unroll
    for (int q = 0; q < 8; q++)
      if (q < left) p[q] = (Out)f[q];
  }
}

}  // namespace q4k
