// C ABI of the paged 8-bit caches (declarations and contract:
// include/kvcache.h); arguments are validated as in nvfp4_api.hip.
#include "../../include/kvcache.h"

#include <hip/hip_runtime.h>

#include <utility>

#include "api_common.hpp"
#include "fp8_kernels.hpp"

namespace {

using namespace nvfp4;

constexpr int64_t kMaxDim = 1024, kMaxHeads = 65536, kMaxElements = (int64_t)1 << 44;
constexpr int64_t kInt32 = (int64_t)1 << 31;

int tensor_sizes(const kv8_tensor& c, const kv8_places& p) {
  if (c.dim <= 0 || c.dim % 16 != 0 || c.token_stride < 0 || c.head_stride < 0) return NVFP4_ERR_SHAPE;
  if (c.dim > kMaxDim) return NVFP4_ERR_UNSUPPORTED;
  const int64_t rows = p.page_size * p.heads;  // < 2^47
  if (c.code_stride < rows * c.dim || c.scale_stride < rows) return NVFP4_ERR_SHAPE;
  if (!mul_ok(p.pages, c.code_stride) || !mul_ok(p.pages, c.scale_stride) || !mul_ok(p.tokens, c.token_stride) ||
      !mul_ok(p.heads, c.head_stride))
    return NVFP4_ERR_SHAPE;
  if (p.tokens * p.heads > kMaxElements / c.dim) return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}

// Rows of an output [tokens, heads, dim] that share no element: the wider of the
// two strides spans all of the narrower one's rows.  (Products fit: tensor_sizes.)
bool rows_apart(const kv8_tensor& c, const kv8_places& p) {
  int64_t s0 = p.tokens > 1 ? c.token_stride : INT64_MAX, s1 = p.heads > 1 ? c.head_stride : INT64_MAX;
  int64_t n1 = p.heads;
  if (s0 < s1) std::swap(s0, s1), n1 = p.tokens;
  return s1 >= c.dim && (s0 == INT64_MAX || s0 - c.dim >= (n1 - 1) * s1);
}

int run(const kv8_tensor* keys, const kv8_tensor* values, const kv8_places* places, int dtype, int q_dtype, bool write,
        void* stream) {
  if (!keys || !values || !places) return NVFP4_ERR_NULL;
  const kv8_places& p = *places;
  const kv8_tensor* both[2] = {keys, values};
  const bool empty = p.tokens == 0 || p.heads == 0;
  if (!empty) {
    for (const kv8_tensor* c : both)
      if (!c->rows || (p.pages > 0 && (!c->codes || !c->scales))) return NVFP4_ERR_NULL;
    if (!p.cu || (p.seqs > 0 && p.table_width > 0 && !p.page_table)) return NVFP4_ERR_NULL;
  }
  if (dtype != NVFP4_F32 && dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
  if (q_dtype != INT4_I8 && q_dtype != INT4_E4M3) return NVFP4_ERR_DTYPE;
  if (p.seqs < 0 || p.table_width < 0 || p.tokens < 0 || p.heads < 0 || p.pages < 0 || p.page_size <= 0)
    return NVFP4_ERR_SHAPE;
  if (p.seqs >= kInt32 || p.table_width >= kInt32 || p.tokens >= kInt32 || p.pages >= kInt32 || p.page_size >= kInt32 ||
      p.heads > kMaxHeads)
    return NVFP4_ERR_UNSUPPORTED;
  for (const kv8_tensor* c : both)
    if (const int st = tensor_sizes(*c, p); st != NVFP4_OK) return st;
  if (empty) return NVFP4_OK;
  for (const kv8_tensor* c : both)
    if (!write && !rows_apart(*c, p)) return NVFP4_ERR_SHAPE;
  const int64_t unit = dtype == NVFP4_BF16 ? 8 : 4;
  for (const kv8_tensor* c : both)
    if (!aligned(c->rows, 16) || c->token_stride % unit != 0 || c->head_stride % unit != 0 || !aligned(c->codes, 16) ||
        c->code_stride % 16 != 0 || !aligned(c->scales, 4))
      return NVFP4_ERR_ALIGN;
  if (!aligned(p.cu, 4) || !aligned(p.starts, 4) || !aligned(p.page_table, 4)) return NVFP4_ERR_ALIGN;
  if (p.seqs == 0) return NVFP4_OK;  // no row belongs to a sequence
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (const int st = stream_status(s); st != NVFP4_OK) return st;
  clear_error();
  return launch_status(launch_kv8(*keys, *values, p, dtype == NVFP4_BF16, q_dtype == INT4_E4M3, write, s));
}

}  // namespace

extern "C" {

int kv8_write(const kv8_tensor* keys, const kv8_tensor* values, const kv8_places* places, int dtype, int q_dtype,
              void* stream) {
  return run(keys, values, places, dtype, q_dtype, true, stream);
}

int kv8_read(const kv8_tensor* keys, const kv8_tensor* values, const kv8_places* places, int dtype, int q_dtype,
             void* stream) {
  return run(keys, values, places, dtype, q_dtype, false, stream);
}

}  // extern "C"
