// C ABI of the group-scaled 4-bit weight path (declarations and the contract
// of every entry point: include/int4.h).  As in nvfp4_api.hip, arguments are
// validated without touching the HIP runtime, then the kernels are launched
// on the caller's stream.
#include "../../include/int4.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "api_common.hpp"
#include "int4_kernels.hpp"

namespace {

using namespace nvfp4;

// Rows of codes are addressed by 32-bit buffer offsets: 64 rows of 2^24
// codes are 2^29 bytes, 16 rows of 2^24 bf16 activations as well.
constexpr int64_t kMaxCols = (int64_t)1 << 24;
// A launch counts its threads in 32 bits: 2^22 workgroups of 64 rows.
constexpr int64_t kMaxN = (int64_t)1 << 28;
constexpr int64_t kMaxNormCols = 65536;

bool group_ok(int group) { return group == 32 || group == 64 || group == 128; }

// Sizes of a packed weight [rows, cols].
int weight_check(int64_t rows, int64_t cols, int group) {
  if (rows < 0 || cols < 0 || !mul_ok(rows, cols)) return NVFP4_ERR_SHAPE;
  if (cols % 16 != 0) return NVFP4_ERR_SHAPE;
  if (cols % 32 != 0 || cols > kMaxCols || !group_ok(group)) return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}

int gemv_common(const Int4Act& x, const Int4Weight& w, int64_t M, int64_t N, int64_t K, void* y, int y_dtype,
                void* stream) {
  const bool empty = M == 0 || N == 0;  // reads no pointer
  if (!empty && (!x.x || !w.codes || !w.scales || !y || (x.type != Act::kBf16 && !x.scales))) return NVFP4_ERR_NULL;
  if (y_dtype != NVFP4_F32 && y_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
  if (M < 0 || !mul_ok(M, K) || !mul_ok(M, N)) return NVFP4_ERR_SHAPE;
  if (const int st = weight_check(N, K, w.group); st != NVFP4_OK) return st;
  if (M > 16 || K == 0 || N > kMaxN) return NVFP4_ERR_UNSUPPORTED;
  if (empty) return NVFP4_OK;
  if (!aligned(x.x, 16) || !aligned(w.codes, 16) || !aligned(w.scales, 2) || !aligned(y, 4) || !aligned(x.scales, 4))
    return NVFP4_ERR_ALIGN;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (const int st = stream_status(s); st != NVFP4_OK) return st;
  clear_error();
  return launch_status(launch_int4_gemv(x, w, M, N, K, y, y_dtype == NVFP4_BF16, s));
}

}  // namespace

extern "C" {

int int4_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int group, uint8_t* codes, void* scales,
                  uint8_t* zeros, void* stream) {
  const bool empty = rows == 0 || cols == 0;
  if (!empty && (!x || !codes || !scales)) return NVFP4_ERR_NULL;
  if (x_dtype != NVFP4_F32 && x_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
  if (const int st = weight_check(rows, cols, group); st != NVFP4_OK) return st;
  if (empty) return NVFP4_OK;
  if (!aligned(x, 16) || !aligned(codes, 4) || !aligned(scales, 2)) return NVFP4_ERR_ALIGN;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (const int st = stream_status(s); st != NVFP4_OK) return st;
  clear_error();
  return launch_status(launch_int4_quantize(x, x_dtype == NVFP4_BF16, rows, cols, group, codes,
                                            reinterpret_cast<uint16_t*>(scales), zeros, s));
}

int int4_dequant(const uint8_t* codes, const void* scales, const uint8_t* zeros, int64_t rows, int64_t cols, int group,
                 void* out, int out_dtype, void* stream) {
  const bool empty = rows == 0 || cols == 0;
  if (!empty && (!codes || !scales || !out)) return NVFP4_ERR_NULL;
  if (out_dtype != NVFP4_F32 && out_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
  if (const int st = weight_check(rows, cols, group); st != NVFP4_OK) return st;
  if (empty) return NVFP4_OK;
  if (!aligned(codes, 4) || !aligned(scales, 2) || !aligned(out, 16)) return NVFP4_ERR_ALIGN;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (const int st = stream_status(s); st != NVFP4_OK) return st;
  clear_error();
  const Int4Weight w{codes, reinterpret_cast<const uint16_t*>(scales), zeros, group};
  return launch_status(launch_int4_dequant(w, rows, cols, out, out_dtype == NVFP4_BF16, s));
}

int int4_gemv_w4a16(const void* x, const uint8_t* codes, const void* scales, const uint8_t* zeros, int group,
                    int64_t M, int64_t N, int64_t K, void* y, int y_dtype, void* stream) {
  return gemv_common({x, Act::kBf16, nullptr, false},
                     {codes, reinterpret_cast<const uint16_t*>(scales), zeros, group}, M, N, K, y, y_dtype, stream);
}

int int4_gemv_w4a8(const void* x, int x_dtype, const float* x_scales, int x_group, const uint8_t* codes,
                   const void* scales, const uint8_t* zeros, int group, int64_t M, int64_t N, int64_t K, void* y,
                   int y_dtype, void* stream) {
  if (x_dtype != INT4_I8 && x_dtype != INT4_E4M3) return NVFP4_ERR_DTYPE;
  if (x_group != 0 && x_group != group) return NVFP4_ERR_UNSUPPORTED;
  return gemv_common({x, x_dtype == INT4_I8 ? Act::kI8 : Act::kE4m3, x_scales, x_group != 0},
                     {codes, reinterpret_cast<const uint16_t*>(scales), zeros, group}, M, N, K, y, y_dtype, stream);
}

int int4_rmsnorm_quant8(const void* x, int x_dtype, int64_t x_stride, const void* residual, int res_dtype,
                        int64_t res_stride, const void* weight, int w_dtype, double eps, int64_t rows, int64_t cols,
                        int group, int q_dtype, void* codes, float* scales, void* residual_out, void* stream) {
  const bool empty = rows == 0;
  if (!empty && (!x || !codes || !scales || (residual && !residual_out))) return NVFP4_ERR_NULL;
  if (x_dtype != NVFP4_F32 && x_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
  if (residual && res_dtype != x_dtype && res_dtype != NVFP4_F32) return NVFP4_ERR_DTYPE;
  if (weight && w_dtype != NVFP4_F32 && w_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
  if (q_dtype != INT4_I8 && q_dtype != INT4_E4M3) return NVFP4_ERR_DTYPE;
  if (!(eps >= 0.0) || std::isinf(eps)) return NVFP4_ERR_FLAGS;
  if (rows < 0 || cols <= 0 || cols % 16 != 0) return NVFP4_ERR_SHAPE;
  if (x_stride < cols || !mul_ok(rows, x_stride)) return NVFP4_ERR_SHAPE;
  if (residual && (res_stride < cols || !mul_ok(rows, res_stride))) return NVFP4_ERR_SHAPE;
  if (cols > kMaxNormCols || (group != 0 && !group_ok(group))) return NVFP4_ERR_UNSUPPORTED;
  if (empty) return NVFP4_OK;
  const auto rows_ok = [](const void* p, int dtype, int64_t stride) {
    return aligned(p, 16) && stride % (dtype == NVFP4_BF16 ? 8 : 4) == 0;
  };
  if (!rows_ok(x, x_dtype, x_stride) || (residual && !rows_ok(residual, res_dtype, res_stride)) ||
      (residual && !aligned(residual_out, 16)) || !aligned(weight, 16) || !aligned(codes, 8) || !aligned(scales, 4))
    return NVFP4_ERR_ALIGN;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (const int st = stream_status(s); st != NVFP4_OK) return st;
  clear_error();
  const NormArgs a{x, residual, weight, codes, scales, residual ? residual_out : nullptr, rows, x_stride, res_stride,
                   (int)cols, group, eps, x_dtype == NVFP4_BF16, residual && res_dtype == NVFP4_BF16,
                   weight && w_dtype == NVFP4_BF16, q_dtype == INT4_E4M3};
  return launch_status(launch_rmsnorm_quant8(a, s));
}

}  // extern "C"
