/*
 * fp8.h -- C ABI of the MI355X (gfx950) library for 8-bit layers: FP8 weights
 * with a scale for each 128 x 128 block and 8-bit activations with a scale
 * for each group of columns (in libnvfp4.so, beside nvfp4.h and int4.h):
 *   - weight quantizer fp8_quantize;
 *   - activation quantizer fp8_quantize_act, of a tensor or of SiLU(gate) x
 *     (a gated MLP's middle); int4_rmsnorm_quant8 with groups of 128 and E4M3
 *     is the third source of the product's activations;
 *   - product fp8_gemm of any number of rows.
 *
 * Format: E4M3 ("fn": bias 7, max 448, no infinities), one byte an element,
 * row-major.
 *   - a weight W [N, K] has fp32 scales [ceil(N / 128), ceil(K / 128)], one
 *     for each block of 128 rows and 128 columns (the last ones may be short);
 *     W^ = scale * code;
 *   - activations x [M, K] have fp32 scales [M, ceil(K / group)], one for each
 *     row and group of columns (the last may be short); x^ = scale * code. The
 *     product takes groups of 128.
 * A scale is fp32(max|v| / Q) of the values v it serves, the quotient exact up
 * to its one rounding and Q = 448 (E4M3) or 127 (INT8); 1.0 where that is 0. A
 * code is the nearest E4M3 or INT8 value to v / scale (exact quotient), ties
 * to even.
 *
 * Statuses and conventions are nvfp4.h's, as in int4.h: device pointers of the
 * current device, calls asynchronous on `stream`, nothing allocated, every
 * argument checked before a launch, NVFP4_ERR_CAPTURE on a stream that is being
 * captured, NULL pointers accepted where a call reads and writes nothing,
 * non-finite inputs a caller error (outputs unspecified). No call needs a
 * workspace, and none keeps state: calls on different streams are independent.
 * No output may overlap an input. nvfp4_version() counts nvfp4.h's interface
 * and did not change with these entry points: look them up by symbol.
 */
#ifndef FP8_H_
#define FP8_H_

#include <stddef.h>
#include <stdint.h>

#include "int4.h" /* INT4_I8, INT4_E4M3 */

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fp8_quantize -- codes and block scales of a weight.
 *   x      [rows, cols] of x_dtype (NVFP4_F32 or NVFP4_BF16), rows x_stride
 *          elements apart
 *   codes  [rows, cols], scales fp32 [ceil(rows/128), ceil(cols/128)]
 * cols % 16 != 0, x_stride < cols: NVFP4_ERR_SHAPE; cols > 2^24:
 * NVFP4_ERR_UNSUPPORTED. x and its rows 16-byte aligned, codes 8, scales 4.
 */
int fp8_quantize(const void* x, int x_dtype, int64_t x_stride, int64_t rows, int64_t cols, uint8_t* codes,
                 float* scales, void* stream);

/*
 * fp8_quantize_act -- 8-bit codes and group scales of activations.
 *   y[r, c] = x[r, c], or with a gate x[r, c] g / (1 + exp(-g)), g = gate[r, c]
 *   (never rounded to 16 or 32 bits: a code or scale is decided by the
 *   definition above, short of values within 2^-44 of a border between two
 *   codes, relative, which fp64 cannot tell from it; of these two calls of
 *   different sizes may take the one and the other, since large ones have
 *   SiLU from a table)
 *   x      [rows, cols] of x_dtype (NVFP4_F32 or NVFP4_BF16), rows x_stride
 *          elements apart; gate the same, rows gate_stride apart, or NULL
 *          (the two halves of one [rows, 2 cols] product, say)
 *   group  32, 64 or 128 (else NVFP4_ERR_UNSUPPORTED)
 *   codes  [rows, cols] of q_dtype (INT4_I8 or INT4_E4M3), scales fp32 [rows,
 *          ceil(cols / group)], both contiguous
 * cols % 16 != 0, a stride < cols: NVFP4_ERR_SHAPE; cols > 2^24:
 * NVFP4_ERR_UNSUPPORTED. x, gate, their rows and codes 16-byte aligned,
 * scales 4. (A product x g / (1 + exp(-g)) beyond fp32's range whose scale
 * leaves it too is a caller error.)
 */
int fp8_quantize_act(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride, int x_dtype, int64_t rows,
                     int64_t cols, int group, int q_dtype, void* codes, float* scales, void* stream);

/*
 * fp8_gemm -- y = x^ W^^T.
 *   y[m, n] = round(sum_b xs[m, b] ws[n / 128, b] sum_{k in b} x[m, k] w[n, k]),
 *   b the blocks of 128 columns
 *   x [M, K], xs [M, ceil(K/128)], w [N, K], ws [ceil(N/128), ceil(K/128)]
 *   y [M, N] of y_dtype (NVFP4_BF16 or NVFP4_F32), contiguous
 * Products of codes are summed within a block, and blocks among each other, in
 * fp32 in an order that M, N, K and y_dtype fix: the same call gives the same
 * bits. An fp32 y of any size, and a bf16 y of few rows before its rounding, is
 * off by at most (K + 4) 2^-24 of the sum of all terms' magnitudes |x^ w^|. The
 * sums behind a bf16 y of more rows (M > 16 and ceil(M / 32) ceil(N / 16) > 512)
 * also lose up to 7 2^-13 of the largest term of each 8 columns, what the FP8
 * matrix instruction cuts off: less than bf16's rounding of a typical result, but
 * not of one whose terms cancel, and a row's results depend in this on how many
 * rows the call has. Where that matters, ask for an fp32 y.
 * xs ws may leave fp32's range as long as xs ws x w does not.
 * A row of x whose codes or scales are no numbers (behind a padded batch, say)
 * reaches its own row of y only; in a weight they are a caller error.
 * K % 16 != 0: NVFP4_ERR_SHAPE; K == 0, K > 2^22, N > 2^26 or M > 2^31:
 * NVFP4_ERR_UNSUPPORTED. x and w 16-byte aligned, scales and y 4.
 */
int fp8_gemm(const uint8_t* x, const float* x_scales, const uint8_t* w, const float* w_scales, int64_t M, int64_t N,
             int64_t K, void* y, int y_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8_H_ */
