/*
 * q4k_mx.h -- microscaled (MX) operators of libq4k.so: quantisation to and
 * from MXFP4 / MXFP8, the root-mean-square norm that feeds them, the product
 * with MXFP4 weights, and a mixture-of-experts layer of such weights.
 *
 * The contract of q4k.h holds here too: device pointers owned by the caller,
 * validation before anything is launched (dimensions, types and formats,
 * then NULL pointers, then alignment), kernels enqueued on `stream`, no
 * allocation, no synchronisation, no state, no C++ exception; every call is
 * deterministic, its summation order a function of the shapes.  Outputs must
 * not overlap inputs except where said.  A call may be captured into a graph.
 *
 * MX format (OCP Microscaling Formats specification, version 1.0): 32
 * consecutive values of a row form a block with one scale byte s standing for
 * 2^(s-127); s = 255 makes the whole block NaN.  A matrix of n_rows rows and
 * input_dim columns (a multiple of 32) is two arrays, both row-major without
 * padding:
 *   codes   MX_FP4: [n_rows][input_dim/2] bytes, e2m1 values (0, 0.5, 1, 1.5,
 *           2, 3, 4, 6 by the low three bits, sign in bit 3), position 2i in
 *           the low nibble of byte i and 2i+1 in its high nibble;
 *           MX_FP8: [n_rows][input_dim] bytes, e4m3 values (bias 7, largest
 *           448, 0x7F and 0xFF NaN)
 *   scales  [n_rows][input_dim/32] bytes
 */
#ifndef Q4K_MX_H
#define Q4K_MX_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Block formats. */
#define MX_FP4 4
#define MX_FP8 8

/* Types of unpacked values. */
#define MX_F32 0
#define MX_BF16 1
#define MX_F16 2

/* A type or a format is none of the above (the codes of q4k.h otherwise). */
#define Q4K_EINVAL_TYPE (-6)

/*
 * mx_quantize -- rows to blocks: with a = the largest magnitude of a block
 * and e = max(floor(log2 a) - m, -127), m = 2 (MX_FP4) or 8 (MX_FP8), its
 * scale byte is e + 127 and each code is x * 2^-e rounded to nearest even and
 * held at 6 or 448 (the conversion of the MX specification).  A block of
 * zeros has scale byte 0 and codes 0 (-0 keeps its sign); a block that holds
 * a NaN or an infinity has scale byte 255 and codes 0.
 *   x          [n_rows][input_dim] of x_type, 16-byte aligned
 *   n_rows     > 0, below 2^31; input_dim > 0, a multiple of 32, at most 2^24
 *   codes      16-byte aligned, every byte written; scales likewise
 *              (any alignment)
 * Exact: the result is a function of the values alone.
 */
int mx_quantize(const void *x, int x_type, int format, int64_t n_rows, int64_t input_dim,
                uint8_t *codes, uint8_t *scales, void *stream);

/*
 * mx_dequantize -- the values that codes and scales stand for, rounded to
 * y_type (to nearest even; exact for fp32, and for bf16 down to its normal
 * range).
 *   codes      16-byte aligned; scales any alignment
 *   y          [n_rows][input_dim] of y_type, 16-byte aligned
 */
int mx_dequantize(const uint8_t *codes, const uint8_t *scales, int format, int64_t n_rows,
                  int64_t input_dim, void *y, int y_type, void *stream);

/*
 * mx_rmsnorm -- the norm between two layers, with the residual's addition
 * before it and the next product's block format after it:
 *   r = x + residual, rounded to `type`        (r = x where residual is NULL)
 *   h = r * rsqrt(mean(r^2) + eps) * weight    in fp32
 *   residual_out = r, y = h rounded to `type`, codes / scales = the blocks of
 *   h as mx_quantize makes them
 *   x, residual, y, residual_out  [n_rows][input_dim] of `type`, 16-byte
 *              aligned; residual_out may be residual itself (or x)
 *   weight     [input_dim] of `type`, 16-byte aligned
 *   eps        >= 0
 *   residual, residual_out, y may be NULL; codes and scales both NULL leave
 *   the blocks out (format is then not read)
 * The mean is an fp32 sum.
 */
int mx_rmsnorm(const void *x, const void *residual, const void *weight, float eps, int type,
               int64_t n_rows, int64_t input_dim, void *residual_out, void *y, int format,
               uint8_t *codes, uint8_t *scales, void *stream);

/*
 * mxfp4_matmul -- Y[t, o] = sum_k A[t, k] * W[o, k], t < n_tokens, with W in
 * MXFP4 and A in MXFP8 or MXFP4, as gfx950's scaled matrix instructions
 * multiply them; accumulated in fp32 and rounded once to y_type.  One such
 * instruction adds 128 e4m3 products with an error of up to 2^-11 of the
 * largest of them (about 5e-6 of a result's norm on normal data).  With fp32
 * outputs MXFP8 activations take two instructions for each product, without
 * that error; with 16-bit outputs they take one.  The error is then below half
 * a step of most outputs, but not of one whose products cancel: take fp32
 * outputs where that matters.  MXFP4 activations have none of it.
 *   a_codes, a_scales  n_tokens rows of input_dim values in a_format
 *   w_codes, w_scales  output_dim rows of input_dim values in MX_FP4
 *   codes 16-byte aligned, scales any alignment
 *   n_tokens   > 0, at most 2^21; output_dim > 0, at most 2^26; input_dim > 0,
 *              a multiple of 32, at most 2^24
 *   Y          [n_tokens][output_dim] of y_type, aligned to its type
 * A NaN block makes the outputs that use it NaN.
 */
int mxfp4_matmul(const uint8_t *a_codes, const uint8_t *a_scales, int a_format,
                 const uint8_t *w_codes, const uint8_t *w_scales, int64_t n_tokens,
                 int64_t input_dim, int64_t output_dim, void *Y, int y_type, void *stream);

/*
 * mxfp4_moe -- a mixture-of-experts layer for a few tokens, three kernels:
 *   logits[t, e] = sum_k x[t, k] * router[e, k] + router_bias[e]   (fp32)
 *   chosen: the top_k experts of the largest logits (equal ones: the lower
 *   index first; a NaN logit comes after all others)
 *   p = softmax over the chosen logits
 *   h = silu(gate_e x) * (up_e x),  y = sum over the chosen of p_e * down_e h
 *   x, y       [n_tokens][input_dim] of `type`, 16-byte aligned
 *   router     [n_experts][input_dim] of `type`, 16-byte aligned
 *   router_bias  fp32 [n_experts], or NULL
 *   up_codes, up_scales      MXFP4 [n_experts][2*ffn_dim][input_dim], an
 *              expert's rows 0 .. ffn_dim-1 gate, the others up
 *   down_codes, down_scales  MXFP4 [n_experts][input_dim][ffn_dim]
 *   input_dim, ffn_dim  > 0, multiples of 32, at most 2^20
 *   n_experts  1 .. 256; top_k 1 .. min(n_experts, 16); n_tokens > 0, at most
 *              2^21
 *   workspace  mxfp4_moe_workspace_size bytes, 256-byte aligned, of any
 *              content; its content after the call is undefined.  Calls that
 *              share one must not overlap in time.
 * What lies between x and y, for finite x and h below 2^127:
 *   logits  fp32 sums, off by up to (input_dim / 256 + 24) 2^-23 of the sum of
 *           |x| |router| and |bias|; of experts whose logits lie closer, either
 *           may be chosen
 *   x       enters the products as one (bf16), two (fp16) or three (fp32) bf16
 *           values that add up to it
 *   h       enters as three bf16 values for fp32, which add up to it, and as
 *           two for bf16 and fp16, off by up to 2^-17 of each |h| before the
 *           sum over ffn_dim
 *   weights e2m1 times their block's scale, exact in bf16 for scale bytes up to
 *           252, as mx_quantize makes them (253: 4 and 6 are infinite, 254: 2
 *           and above); 255 makes the outputs that use the block NaN
 *   sums    fp32
 * An expert's weights are read once for up to 16 of its tokens (8 where
 * n_tokens * top_k is at most 2 * n_experts), and again for more.  At most 64
 * tokens run at a time, more loop over them and read the experts' weights
 * again: the call is for few tokens.  Fewer run at a time from 129 experts
 * on (8192 / n_experts), and where top_k * max(input_dim, ffn_dim) passes 5.5
 * million (2^31 / 6 of it, so that a group's slots stay within 31-bit offsets).
 * workspace_bytes too small gives Q4K_ESCRATCH.
 */
int64_t mxfp4_moe_workspace_size(int64_t n_tokens, int64_t input_dim, int64_t ffn_dim,
                                 int64_t n_experts, int64_t top_k);
int mxfp4_moe(const void *x, int type, const void *router, const float *router_bias,
              const uint8_t *up_codes, const uint8_t *up_scales, const uint8_t *down_codes,
              const uint8_t *down_scales, int64_t n_tokens, int64_t input_dim, int64_t ffn_dim,
              int64_t n_experts, int64_t top_k, void *y, void *workspace, int64_t workspace_bytes,
              void *stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4K_MX_H */
