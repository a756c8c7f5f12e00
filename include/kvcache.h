/*
 * kvcache.h -- C ABI of the MI355X (gfx950) library for paged 8-bit caches of
 * keys and values (in libnvfp4.so, beside nvfp4.h, int4.h and fp8.h):
 *   - kv8_write quantizes new tokens' keys and values as it writes them;
 *   - kv8_read reads ranges of sequences back as fp32 or bf16.
 *
 * Format: a cache of one tensor (keys, or values) is codes [pages, page_size,
 * heads, dim] of one byte an element, INT8 or E4M3, and fp32 scales [pages,
 * page_size, heads], one for each token and head: the value is scale * code.
 * A page's codes and its scales are contiguous; pages are code_stride bytes
 * and scale_stride floats apart (a keys' and a values' cache may be slices of
 * one allocation). scale = fp32(max|v| / Q) over the head's dim elements,
 * Q = 127 or 448, the quotient exact up to its one rounding, 1.0 where that is
 * 0; code = nearest value to v / scale (exact quotient), ties to even.
 *
 * Places: the calls work on `tokens` rows that belong to `seqs` sequences.
 * Rows cu[b] .. cu[b + 1] - 1 belong to sequence b (int32 cu [seqs + 1], none
 * negative, non-decreasing); row t is the sequence's position p = starts[b] + t - cu[b]
 * (int32 starts [seqs], or NULL for 0), which lies in row p % page_size of page
 * page_table[b, p / page_size] (int32 [seqs, table_width], contiguous). Rows
 * before cu[0] and from cu[seqs] on belong to no sequence. A position below 0
 * or at or past table_width * page_size, and a page number below 0 or at or
 * past `pages`, is no place: kv8_write writes nothing for it, kv8_read writes
 * zeros. Two rows with the same place in one kv8_write (a page that two
 * sequences share) leave that place unspecified, and no other.
 *
 * Statuses and conventions are nvfp4.h's, as in int4.h: device pointers of the
 * current device, calls asynchronous on `stream`, nothing allocated, every
 * argument checked before a launch (what the tables hold is checked by the
 * kernels as above), NVFP4_ERR_CAPTURE on a stream that is being captured,
 * non-finite inputs a caller error (the codes and scale of that token and head
 * are unspecified). No call needs a workspace, and none keeps state. Each call
 * takes keys and values together; dim may differ between them.
 */
#ifndef KVCACHE_H_
#define KVCACHE_H_

#include <stddef.h>
#include <stdint.h>

#include "int4.h" /* INT4_I8, INT4_E4M3 */

#ifdef __cplusplus
extern "C" {
#endif

/* One tensor of a cache and the rows that a call writes to it or reads from it. */
typedef struct {
  void* codes;          /* 16-byte aligned */
  float* scales;        /* 4-byte aligned */
  int64_t code_stride;  /* bytes from page to page, a multiple of 16 */
  int64_t scale_stride; /* floats from page to page */
  void* rows;           /* [tokens, heads, dim]: kv8_write's input, kv8_read's output, 16-byte aligned */
  int64_t token_stride; /* elements from token to token, and head to head; bytes a multiple of 16 */
  int64_t head_stride;
  int64_t dim;          /* a multiple of 16, at most 1024 */
} kv8_tensor;

/* Where the rows belong. */
typedef struct {
  const int32_t* page_table; /* [seqs, table_width] */
  const int32_t* cu;         /* [seqs + 1] */
  const int32_t* starts;     /* [seqs], or NULL */
  int64_t seqs, table_width, tokens, heads, pages, page_size;
} kv8_places;

/*
 * kv8_write -- quantizes rows of dtype (NVFP4_F32 or NVFP4_BF16) into a cache
 * of q_dtype (INT4_I8 or INT4_E4M3); every place that no row has is left as it
 * was.
 * kv8_read -- writes rows of dtype, fp32(scale * code) or that rounded to bf16
 * (nearest, ties to even); rows of no sequence are left as they were.
 * tokens = 0 or heads = 0 does nothing and reads no pointer but the structs.
 * Negative sizes, dim % 16 != 0, dim <= 0, page_size <= 0, page strides shorter
 * than a page, negative token or head strides: NVFP4_ERR_SHAPE; dim > 1024,
 * heads > 65536, seqs, table_width, tokens, pages or page_size >= 2^31, or more
 * than 2^44 elements of rows: NVFP4_ERR_UNSUPPORTED. No output may overlap an
 * input or another output; rows of kv8_read that overlap each other are
 * NVFP4_ERR_SHAPE (so are rows of whose two strides neither spans all that the
 * other one counts).
 */
int kv8_write(const kv8_tensor* keys, const kv8_tensor* values, const kv8_places* places, int dtype, int q_dtype,
              void* stream);
int kv8_read(const kv8_tensor* keys, const kv8_tensor* values, const kv8_places* places, int dtype, int q_dtype,
             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVCACHE_H_ */
