// mx_common.h -- device helpers of the microscaled (MX) kernels: typed loads
// and stores, the block scale, and the conversions between fp32 and the
// e2m1 / e4m3 codes (include/q4k_mx.h has the format).
#pragma once

#include "device_common.h"
#include "q4k_mx.h"

namespace q4k {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));  // one bf16 MFMA operand
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));  // one f8f6f4 MFMA operand

constexpr int kMxBlock = 32;

// Storage of a value type: MX_F32, MX_BF16 or MX_F16.
template <int T> struct MxStore;
template <> struct MxStore<MX_F32> { typedef float type; };
template <> struct MxStore<MX_BF16> { typedef __bf16 type; };
template <> struct MxStore<MX_F16> { typedef _Float16 type; };

// Eight consecutive values as they lie in memory (32 or 16 bytes).
template <int T> struct Raw8 { u32x4 v; };
template <> struct Raw8<MX_F32> { u32x4 v, w; };

template <int T> __device__ __forceinline__ Raw8<T> load_raw8(const void *p, int64_t chunk) {
  const u32x4 *q = reinterpret_cast<const u32x4 *>(p);
  Raw8<T> r;
  if constexpr (T == MX_F32) {
    r.v = q[2 * chunk];
    r.w = q[2 * chunk + 1];
  } else {
    r.v = q[chunk];
  }
  return r;
}

template <int T> __device__ __forceinline__ void raw8_to_f32(const Raw8<T> &r, float (&f)[8]) {
  if constexpr (T == MX_F32) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[i] = __builtin_bit_cast(float, (uint32_t)r.v[i]);
      f[4 + i] = __builtin_bit_cast(float, (uint32_t)r.w[i]);
    }
  } else if constexpr (T == MX_BF16) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[2 * i] = __builtin_bit_cast(float, (uint32_t)r.v[i] << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, (uint32_t)r.v[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const half2_t h = as_h2(r.v[i]);
      f[2 * i] = (float)h.x;
      f[2 * i + 1] = (float)h.y;
    }
  }
}

// Rounds to nearest even to the type (the identity for fp32).
template <int T> __device__ __forceinline__ Raw8<T> f32_to_raw8(const float (&f)[8]) {
  Raw8<T> r;
  if constexpr (T == MX_F32) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      r.v[i] = __builtin_bit_cast(uint32_t, f[i]);
      r.w[i] = __builtin_bit_cast(uint32_t, f[4 + i]);
    }
  } else if constexpr (T == MX_BF16) {
#pragma unroll
    for (int i = 0; i < 4; i++)
      r.v[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)f[2 * i], (__bf16)f[2 * i + 1]});
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      r.v[i] = as_u32h(half2_t{(_Float16)f[2 * i], (_Float16)f[2 * i + 1]});
  }
  return r;
}

// ONCE: past the caches (the non-temporal hint), for outputs that are larger
// than what the L2s keep until their next use.
template <int T, bool ONCE = false>
__device__ __forceinline__ void store_raw8(void *p, int64_t chunk, const Raw8<T> &r) {
  u32x4 *q = reinterpret_cast<u32x4 *>(p) + (T == MX_F32 ? 2 * chunk : chunk);
  if constexpr (ONCE) {
    __builtin_nontemporal_store(r.v, q);
    if constexpr (T == MX_F32) __builtin_nontemporal_store(r.w, q + 1);
  } else {
    *q = r.v;
    if constexpr (T == MX_F32) q[1] = r.w;
  }
}

// A block's scale byte from the bits of its largest magnitude: the biased
// exponent field is 127 + floor(log2 a) for every normal a, so the byte is
// that field less 2 (e2m1) or 8 (e4m3), at least 0 (subnormal a too); the
// bits of an infinity or a NaN give 255.
template <int FMT> __device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - (FMT == MX_FP4 ? 2 : 8);
  return amax_bits >= 0x7F800000u ? 255u : (uint32_t)(e > 0 ? e : 0);
}

// 2^(s - 127) as fp32: 2^-127 (s = 0) is subnormal, 255 is NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t s) {
  const uint32_t b = s == 0 ? 0x00400000u : (s == 255 ? 0x7FC00000u : s << 23);
  return __builtin_bit_cast(float, b);
}

// The largest |f| of the 32 values that four neighbouring lanes hold eight
// each, as bits: the integer order of the magnitudes' bits is their order,
// with infinities and NaNs on top.
__device__ __forceinline__ uint32_t block_amax_bits(const float (&f)[8]) {
  uint32_t b = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint32_t a = __builtin_bit_cast(uint32_t, f[i]) & 0x7FFFFFFFu;
    b = a > b ? a : b;
  }
  b = max_dpp_step<0xB1>(b);  // quad_perm [1,0,3,2]
  return max_dpp_step<0x4E>(b);  // quad_perm [2,3,0,1]
}

// Eight values as codes under scale byte s: 4 bytes (e2m1, the first dword)
// or 8 (e4m3).  The division by 2^(s-127) is a multiplication by the power
// with exponent field 254 - s (normal, or 2^127 for s = 0), exact unless the
// quotient is below 2^-126 and rounds to zero anyway.  The e2m1 conversion
// saturates by itself; e4m3 gives NaN above 464, so the quotients are held at
// 448 first.  A NaN block gets zero codes.
template <int FMT>
__device__ __forceinline__ u32x2 mx_encode8(const float (&f)[8], uint32_t s) {
  const float inv = __builtin_bit_cast(float, (254u - (s < 254u ? s : 253u)) << 23);
  uint32_t lo = 0, hi = 0;
  if constexpr (FMT == MX_FP4) {
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, f[0] * inv, f[1] * inv, 1.0f, 0);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, f[2] * inv, f[3] * inv, 1.0f, 1);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, f[4] * inv, f[5] * inv, 1.0f, 2);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, f[6] * inv, f[7] * inv, 1.0f, 3);
  } else {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __builtin_amdgcn_fmed3f(f[i] * inv, -448.0f, 448.0f);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], (int)lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], (int)hi, true);
  }
  return s == 255 ? u32x2{0, 0} : u32x2{lo, hi};
}

template <int FMT> __device__ __forceinline__ void mx_decode8(u32x2 c, float scale, float (&f)[8]) {
  if constexpr (FMT == MX_FP4) {
#define Q4K_DEC(i)                                                              \
  {                                                                             \
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], 1.0f, i);    \
    f[2 * i] = v[0] * scale;                                                    \
    f[2 * i + 1] = v[1] * scale;                                                \
  }
    Q4K_DEC(0) Q4K_DEC(1) Q4K_DEC(2) Q4K_DEC(3)
#undef Q4K_DEC
  } else {
#define Q4K_DEC(i, h)                                                           \
  {                                                                             \
    const f32x2 v = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], h);              \
    f[4 * i + 2 * h] = v[0] * scale;                                            \
    f[4 * i + 2 * h + 1] = v[1] * scale;                                        \
  }
    Q4K_DEC(0, 0) Q4K_DEC(0, 1) Q4K_DEC(1, 0) Q4K_DEC(1, 1)
#undef Q4K_DEC
  }
}

// Rounds a value to a type and stores it.
template <int T> __device__ __forceinline__ void store_value(void *p, int64_t i, float v) {
  reinterpret_cast<typename MxStore<T>::type *>(p)[i] = (typename MxStore<T>::type)v;
}

// Keeps the registers of an operand alive until d is written.
template <int F> __device__ __forceinline__ void keep_operand(f32x4 &d, i32x8 v) {
  if constexpr (F == MX_FP4) {
    const i32x4 lo = {v[0], v[1], v[2], v[3]};
    asm("" : "+v"(d) : "v"(lo));
  } else {
    asm("" : "+v"(d) : "v"(v));
  }
}

// D += A * B over 16 rows x 16 columns x 128 positions on the scaled matrix
// instruction; A in format AF, B in BF.  Lane l holds row (column) l % 16 of
// its operand and, with g = l / 16, the positions
//   MX_FP4: 32g .. 32g+31 (16 bytes in the first four dwords)
//   MX_FP8: 16g .. 16g+15 and 64+16g .. 64+16g+15 (the low and the high half)
// and the scale byte of block g (positions 32g .. 32g+31) of its row in
// byte J of sa (sb); D has column l % 16, rows 4g .. 4g+3.  The instruction
// gives wrong sums when D lies on registers of A or B (seen with this
// compiler, which allows it where an operand dies there): keep_operand holds
// both until D is written, at no instruction.
template <int AF, int BF, int J = 0>
__device__ __forceinline__ f32x4 mfma_scaled(i32x8 a, i32x8 b, f32x4 d, int sa, int sb) {
  d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, d, AF == MX_FP4 ? 4 : 0,
                                                       BF == MX_FP4 ? 4 : 0, J, sa, J, sb);
  keep_operand<AF>(d, a);
  keep_operand<BF>(d, b);
  return d;
}

// e4m3 codes as two operands that add up to them: the values of 2 and above
// and the ones below.  The scaled instruction adds the products of an e4m3
// operand in a window of limited width (measured on random codes: off by up
// to 2^-11 of the largest product, 5e-5 of a result's norm; 5e-6 on normal
// data), which half of e4m3's exponents fits: the two parts together come out
// with fp32's error (no bit off within blocks of one scale).  e2m1 with e2m1
// is exact as it is.
__device__ __forceinline__ void split_e4m3(i32x8 v, i32x8 &high, i32x8 &low) {
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint32_t b = (uint32_t)v[i], t = b & 0x40404040u;  // exponent field 8 and above
    const uint32_t m = (t << 1) - (t >> 6);                  // 0x7F in those bytes
    high[i] = (int)(b & (m | 0x80808080u));
    low[i] = (int)(b & ~m);
  }
}

// The product with all of fp32's accuracy (EXACT) or as the instruction adds.
template <int AF, int BF, bool EXACT, int J = 0>
__device__ __forceinline__ f32x4 mfma_mx(i32x8 a, i32x8 b, f32x4 d, int sa, int sb) {
  if constexpr (EXACT && BF == MX_FP8) {
    i32x8 high, low;
    split_e4m3(b, high, low);
    d = mfma_scaled<AF, BF, J>(a, low, d, sa, sb);
    return mfma_scaled<AF, BF, J>(a, high, d, sa, sb);
  } else {
    return mfma_scaled<AF, BF, J>(a, b, d, sa, sb);
  }
}

}  // namespace q4k
