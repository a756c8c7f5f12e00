// Internal launchers of the 8-bit layer kernels (host side).  Arguments are
// validated by the C ABI layers (fp8_api.hip, kvcache_api.hip) before any of
// these is called.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/kvcache.h"

namespace nvfp4 {

struct ActArgs {
  const void* x;
  const void* gate;  // nullptr: none
  void* codes;
  float* scales;
  int64_t rows, x_stride, gate_stride;
  int cols, group;
  bool bf16, e4m3;
};
struct Fp8Product {
  const uint8_t* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  int64_t M;
  int N, K;
  void* y;
  int64_t y_stride;  // N of the whole product: a launch may have some of its columns
  bool bf16;
  int group = 0;  // of the launch: tiles of x that an XCD's stretch of tiles covers
};

hipError_t launch_fp8_quantize(const void* x, bool bf16, int64_t stride, int64_t rows, int64_t cols, uint8_t* codes,
                               float* scales, hipStream_t stream);
hipError_t launch_fp8_quantize_act(const ActArgs& a, hipStream_t stream);
hipError_t launch_fp8_gemm(const Fp8Product& p, hipStream_t stream);
hipError_t launch_kv8(const kv8_tensor& keys, const kv8_tensor& values, const kv8_places& places, bool bf16, bool e4m3,
                      bool write, hipStream_t stream);

}  // namespace nvfp4
