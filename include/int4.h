/*
 * int4.h -- C ABI of the MI355X (gfx950) library for group-scaled 4-bit
 * integer weights and 8-bit activations (in libnvfp4.so, beside nvfp4.h):
 *   - weight quantizer int4_quantize and its inverse int4_dequant;
 *   - decode products int4_gemv_w4a16 (bf16 activations) and
 *     int4_gemv_w4a8 (INT8 or FP8 activations with scales);
 *   - int4_rmsnorm_quant8: residual addition, RMS norm and 8-bit output with
 *     scales, the activations int4_gemv_w4a8 reads.
 *
 * Format (the INT4 "g128" weights of "Cuantizacion para serving", sections
 * on GPTQ and AWQ, about 4.25 bits a weight): a tensor W [rows, cols]
 * (row-major, cols = the reduction dimension K) is cut along cols into groups
 * of `group` = 32, 64 or 128 elements, G = ceil(cols / group) a row (the last
 * group of a row may be short):
 *   - scales [rows, G] bf16; zeros [rows, G] uint8 in 0..15, or NULL for a
 *     symmetric tensor, whose zero point is 8 everywhere;
 *   - W^ = scale * (code - zero), code in 0..15;
 *   - codes [rows, cols/2] uint8: byte 4 d + b of a row (b = 0..3) holds the
 *     code of element 8 d + b in its low nibble and of element 8 d + 4 + b in
 *     its high nibble, so that one mask (and one shift) turns a dword into
 *     bytes in element order.
 * 8-bit activations: one byte an element, INT8 (INT4_I8) or FP8 E4M3 "fn"
 * (INT4_E4M3), with fp32 scales [rows, 1], or [rows, ceil(cols / group)] for
 * groups of `group` columns; the value is scale * code.
 *
 * The format is the grouping and arithmetic of such checkpoints, not their
 * files: codes, scales and zero points have this library's own order and types
 * (GPTQ and AWQ files pack int32 words in orders of their own and scale in
 * fp16, three bits more than bf16).  Nothing here reads them; int4_quantize
 * makes a weight from its 16- or 32-bit values.
 *
 * The products take up to 16 rows.  For more, int4_dequant makes a bf16 weight
 * for a library product, and 8-bit activations are scale * code in any tensor
 * library, or the norm is taken in 16 bits.
 *
 * These entry points came to the library at version 1.8.1 without a change of
 * nvfp4_version(), which counts nvfp4.h's interface: look them up by symbol.
 *
 * Statuses and conventions are nvfp4.h's: device pointers of the current
 * device, calls asynchronous on `stream`, nothing allocated, every argument
 * checked before a launch, NVFP4_ERR_CAPTURE on a stream that is being
 * captured, NULL pointers accepted where an empty tensor or product reads
 * and writes nothing, non-finite inputs a caller error (outputs unspecified).
 * No call needs a workspace, and none keeps state: calls on different streams
 * are independent.  Unless said otherwise no output may overlap an input.
 */
#ifndef INT4_H_
#define INT4_H_

#include <stddef.h>
#include <stdint.h>

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit activation types, beside NVFP4_F32 and NVFP4_BF16 */
enum { INT4_I8 = 2, INT4_E4M3 = 3 };

/*
 * int4_quantize -- codes, scales and zero points of a weight.
 *   x      [rows, cols] of x_dtype (NVFP4_F32 or NVFP4_BF16), 16-byte aligned
 *   codes  [rows, cols/2], 4-byte aligned; scales [rows, G] bf16, 2-byte
 *          aligned; zeros [rows, G], or NULL: symmetric
 *   For each group, with rne = nearest integer, ties to even:
 *   symmetric: s = bf16(fp32(max|w| / 7)), code = clamp(rne(w / s), -8, 7) + 8
 *   otherwise: lo = min(0, min w), hi = max(0, max w),
 *              s = bf16(fp32((hi - lo) / 15)), z = clamp(rne(-lo / s), 0, 15),
 *              code = clamp(rne(w / s) + z, 0, 15)
 *   with the quotients exact (decided as if in infinite precision) and the
 *   range (hi - lo) / 15 or max|w| / 7 computed in fp64.  Where s is 0 (a
 *   group of zeros, or of values whose scale rounds to 0) z is 0 and every
 *   code is the zero point.
 * cols % 16 != 0 is NVFP4_ERR_SHAPE; cols % 32 != 0, cols > 2^24 or another
 * group is NVFP4_ERR_UNSUPPORTED.
 */
int int4_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int group, uint8_t* codes, void* scales,
                  uint8_t* zeros, void* stream);

/*
 * int4_dequant -- out = scale * (code - zero), [rows, cols] of out_dtype
 * (NVFP4_F32, exact; or NVFP4_BF16, rounded once to nearest even), 16-byte
 * aligned.  Shapes, alignment and limits as int4_quantize.
 */
int int4_dequant(const uint8_t* codes, const void* scales, const uint8_t* zeros, int64_t rows, int64_t cols, int group,
                 void* out, int out_dtype, void* stream);

/*
 * int4_gemv_w4a16 -- y = x W^^T for bf16 activations (decoding: every weight
 * is read once per call, so the call is bound by memory bandwidth).
 *   y[m, n] = round(sum_g s[n, g] sum_{k in g} x[m, k] (code[n, k] - z[n, g]))
 *   x [M, K] bf16, 16-byte aligned; codes [N, K/2], 16-byte aligned; scales
 *   [N, G], 2-byte aligned; zeros [N, G] or NULL; y [M, N] of y_dtype
 *   (NVFP4_BF16 or NVFP4_F32), 4-byte aligned
 *   0 <= M <= 16; K % 32 == 0, 0 < K <= 2^24; N <= 2^28, otherwise
 *   NVFP4_ERR_UNSUPPORTED (K % 16 != 0: NVFP4_ERR_SHAPE).  fp32 accumulation
 *   in a fixed order (results are reproducible), RNE bf16 output.  A group's
 *   sum is the difference of sum x code and z sum x, then scaled and added: the
 *   fp32 result is off by at most
 *     2^-24 (129 sum_k |x| s (code + z) + (K / 32 + 26) sum_r |t_r|)
 *   with t_r the terms of the sum over runs of 32 elements (short of sums
 *   outside fp32's normal range).
 */
int int4_gemv_w4a16(const void* x, const uint8_t* codes, const void* scales, const uint8_t* zeros, int group,
                    int64_t M, int64_t N, int64_t K, void* y, int y_dtype, void* stream);

/*
 * int4_gemv_w4a8 -- the same product for 8-bit activations with scales.
 *   x        [M, K] of x_dtype (INT4_I8 or INT4_E4M3), 16-byte aligned
 *   x_scales fp32 [M, 1] with x_group 0, or [M, G] with x_group == group;
 *            4-byte aligned (another x_group is NVFP4_ERR_UNSUPPORTED)
 *   y[m, n] = round(sum_g s[n, g] sx[m, g] sum_{k in g} x[m, k] (code - z))
 *   INT8 sums inside a group are exact integers, which leaves only the second
 *   part of the bound above; everything else is fp32.
 *   Arguments and limits otherwise as int4_gemv_w4a16.
 */
int int4_gemv_w4a8(const void* x, int x_dtype, const float* x_scales, int x_group, const uint8_t* codes,
                   const void* scales, const uint8_t* zeros, int group, int64_t M, int64_t N, int64_t K, void* y,
                   int y_dtype, void* stream);

/*
 * int4_rmsnorm_quant8 -- residual addition, RMS norm, 8-bit output.
 *   h = residual ? round_to_res_dtype(fp32(x + residual)) : x
 *   y[r, c] = h[r, c] w[c] / sqrt(sum_c h[r, c]^2 / cols + eps)
 *   scale   = fp32(max|y| / Q) over the row (group 0) or each group of
 *             `group` = 32, 64 or 128 columns (the last may be short);
 *             Q = 127 (INT4_I8) or 448 (INT4_E4M3); 1.0 where that is 0
 *   code    = nearest INT8 (ties to even) or E4M3 value to y / scale
 *   h is what the next layer's residual stream holds, and the norm is of its
 *   rounded value; y is never rounded to 16 bits: products, maxima, sums and
 *   quotients are held in fp64 wherever fp32 would round, underflow or
 *   overflow, so codes and scales are decided by the definition above (short
 *   of quotients within 2^-45 of half way, which fp64 cannot tell from it).
 *   (A weight so large that a scale passes fp32's range is a caller error.)
 *   x        [rows, cols] of x_dtype (NVFP4_F32 or NVFP4_BF16), rows
 *            x_stride elements apart
 *   residual [rows, cols] of res_dtype (x_dtype or NVFP4_F32), rows
 *            res_stride elements apart, or NULL (then res_dtype and
 *            residual_out are not used)
 *   weight   [cols] of w_dtype (NVFP4_F32 or NVFP4_BF16), or NULL for ones
 *   codes    [rows, cols] contiguous; scales fp32 [rows, 1 or ceil(cols/group)]
 *   residual_out [rows, cols] contiguous of res_dtype: h; it may be the
 *            residual or x itself (in place) where type and strides agree
 *   cols % 16 == 0, cols > 0 and strides >= cols (else NVFP4_ERR_SHAPE), cols <=
 *   65536 (NVFP4_ERR_UNSUPPORTED), eps finite and >= 0 (NVFP4_ERR_FLAGS);
 *   pointers and rows 16-byte aligned (codes 8, scales 4).
 */
int int4_rmsnorm_quant8(const void* x, int x_dtype, int64_t x_stride, const void* residual, int res_dtype,
                        int64_t res_stride, const void* weight, int w_dtype, double eps, int64_t rows, int64_t cols,
                        int group, int q_dtype, void* codes, float* scales, void* residual_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* INT4_H_ */
