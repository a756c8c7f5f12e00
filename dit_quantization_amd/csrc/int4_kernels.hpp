// Internal launchers of the group-scaled 4-bit weight and 8-bit activation
// kernels (host side).  Arguments are validated by the C ABI layer
// (int4_api.hip) before any of these is called.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {

// A group-scaled 4-bit weight (layout: include/int4.h); zeros == nullptr: 8.
struct Int4Weight {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  int group;
};
// Activations of a decode product: bf16 (scales == nullptr), INT8 or E4M3.
enum class Act { kBf16, kI8, kE4m3 };
struct Int4Act {
  const void* x;
  Act type;
  const float* scales;
  bool grouped;  // scales [M, G]; otherwise [M, 1]
};
struct NormArgs {
  const void* x;
  const void* residual;  // nullptr: none
  const void* weight;    // nullptr: ones
  void* codes;
  float* scales;
  void* residual_out;
  int64_t rows, x_stride, res_stride;
  int cols, group;  // group 0: one scale per row
  double eps;
  bool x_bf16, res_bf16, w_bf16, e4m3;
};

hipError_t launch_int4_quantize(const void* x, bool bf16, int64_t rows, int64_t cols, int group, uint8_t* codes,
                                uint16_t* scales, uint8_t* zeros, hipStream_t stream);
hipError_t launch_int4_dequant(const Int4Weight& w, int64_t rows, int64_t cols, void* out, bool bf16_out,
                               hipStream_t stream);
hipError_t launch_int4_gemv(const Int4Act& x, const Int4Weight& w, int64_t M, int64_t N, int64_t K, void* y,
                            bool bf16_out, hipStream_t stream);
hipError_t launch_rmsnorm_quant8(const NormArgs& a, hipStream_t stream);

}  // namespace nvfp4
