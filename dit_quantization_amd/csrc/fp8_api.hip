// C ABI of the 8-bit layers (declarations and the contract of every entry
// point: include/fp8.h).  As in nvfp4_api.hip, arguments are validated without
// touching the HIP runtime, then the kernels are launched on the caller's
// stream.
#include "../../include/fp8.h"

#include <hip/hip_runtime.h>

#include "api_common.hpp"
#include "fp8_kernels.hpp"

namespace {

using namespace nvfp4;

constexpr int64_t kMaxCols = (int64_t)1 << 24;
// Panels of 256 rows are addressed by 32-bit buffer offsets: 2^30 bytes.
constexpr int64_t kMaxK = (int64_t)1 << 22;
// Rows of x come in several launches where there are many; a launch counts its
// threads in 32 bits and takes at least 16 of them, 2^22 workgroups of 16 rows
// of the weight.
constexpr int64_t kMaxM = (int64_t)1 << 31;
constexpr int64_t kMaxN = (int64_t)1 << 26;

bool rows_ok(const void* p, int dtype, int64_t stride) {
  return aligned(p, 16) && stride % (dtype == NVFP4_BF16 ? 8 : 4) == 0;
}

int begin(void* stream, hipStream_t* s) {
  *s = reinterpret_cast<hipStream_t>(stream);
  if (const int st = stream_status(*s); st != NVFP4_OK) return st;
  clear_error();
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int fp8_quantize(const void* x, int x_dtype, int64_t x_stride, int64_t rows, int64_t cols, uint8_t* codes,
                 float* scales, void* stream) {
  const bool empty = rows == 0 || cols == 0;
  if (!empty && (!x || !codes || !scales)) return NVFP4_ERR_NULL;
  if (x_dtype != NVFP4_F32 && x_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
  if (rows < 0 || cols < 0 || cols % 16 != 0 || x_stride < cols || !mul_ok(rows, x_stride)) return NVFP4_ERR_SHAPE;
  if (cols > kMaxCols) return NVFP4_ERR_UNSUPPORTED;
  if (empty) return NVFP4_OK;
  if (!rows_ok(x, x_dtype, x_stride) || !aligned(codes, 8) || !aligned(scales, 4)) return NVFP4_ERR_ALIGN;
  hipStream_t s;
  if (const int st = begin(stream, &s); st != NVFP4_OK) return st;
  return launch_status(launch_fp8_quantize(x, x_dtype == NVFP4_BF16, x_stride, rows, cols, codes, scales, s));
}

int fp8_quantize_act(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride, int x_dtype, int64_t rows,
                     int64_t cols, int group, int q_dtype, void* codes, float* scales, void* stream) {
  const bool empty = rows == 0 || cols == 0;
  if (!empty && (!x || !codes || !scales)) return NVFP4_ERR_NULL;
  if (x_dtype != NVFP4_F32 && x_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
  if (q_dtype != INT4_I8 && q_dtype != INT4_E4M3) return NVFP4_ERR_DTYPE;
  if (rows < 0 || cols < 0 || cols % 16 != 0 || x_stride < cols || !mul_ok(rows, x_stride)) return NVFP4_ERR_SHAPE;
  if (gate && (gate_stride < cols || !mul_ok(rows, gate_stride))) return NVFP4_ERR_SHAPE;
  if (cols > kMaxCols || (group != 32 && group != 64 && group != 128)) return NVFP4_ERR_UNSUPPORTED;
  if (empty) return NVFP4_OK;
  if (!rows_ok(x, x_dtype, x_stride) || (gate && !rows_ok(gate, x_dtype, gate_stride)) || !aligned(codes, 16) ||
      !aligned(scales, 4))
    return NVFP4_ERR_ALIGN;
  hipStream_t s;
  if (const int st = begin(stream, &s); st != NVFP4_OK) return st;
  const ActArgs a{x,          gate,  codes,        scales, rows, x_stride, gate_stride, (int)cols, group, x_dtype == NVFP4_BF16,
                  q_dtype == INT4_E4M3};
  return launch_status(launch_fp8_quantize_act(a, s));
}

int fp8_gemm(const uint8_t* x, const float* x_scales, const uint8_t* w, const float* w_scales, int64_t M, int64_t N,
             int64_t K, void* y, int y_dtype, void* stream) {
  const bool empty = M == 0 || N == 0;  // reads no pointer
  if (!empty && (!x || !x_scales || !w || !w_scales || !y)) return NVFP4_ERR_NULL;
  if (y_dtype != NVFP4_F32 && y_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
  if (M < 0 || N < 0 || K < 0 || K % 16 != 0) return NVFP4_ERR_SHAPE;
  if (K == 0 || K > kMaxK || M > kMaxM || N > kMaxN) return NVFP4_ERR_UNSUPPORTED;
  if (empty) return NVFP4_OK;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(y, 4))
    return NVFP4_ERR_ALIGN;
  hipStream_t s;
  if (const int st = begin(stream, &s); st != NVFP4_OK) return st;
  return launch_status(
      launch_fp8_gemm({x, x_scales, w, w_scales, M, (int)N, (int)K, y, N, y_dtype == NVFP4_BF16}, s));
}

}  // extern "C"
