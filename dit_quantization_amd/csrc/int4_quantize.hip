// Group-scaled 4-bit integer weights (format: include/int4.h): the quantizer
// and its inverse.
#include "device_common.hpp"
#include "int4_kernels.hpp"

namespace nvfp4 {

// 8 consecutive elements of row r from column c.
template <bool BF16>
__device__ __forceinline__ void load8(const void* x, int64_t i, float v[8]) {
  if (BF16) {
    const u32x4 u = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(x) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(u[j] << 16);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
  } else {
    const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(x) + i);
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  }
}

// One thread per group.
template <bool BF16>
__global__ __launch_bounds__(256) void int4_quantize_kernel(const void* __restrict__ x, int64_t slots, int64_t G,
                                                            int cols, int group, uint8_t* __restrict__ codes,
                                                            uint16_t* __restrict__ scales,
                                                            uint8_t* __restrict__ zeros) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < slots; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / G;
    const int c0 = (int)(i % G) * group, n = min(group, cols - c0);
    const int64_t base = r * cols + c0;
    float lo = 0.0f, hi = 0.0f, v[8];
    for (int c = 0; c < n; c += 8) {
      load8<BF16>(x, base + c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        lo = fminf(lo, v[j]);
        hi = fmaxf(hi, v[j]);
      }
    }
    const double range = zeros ? ((double)hi - (double)lo) * (1.0 / 15.0) : (double)fmaxf(hi, -lo) * (1.0 / 7.0);
    const uint32_t sb = f32_to_bf16_bits((float)range);
    const double s = (double)bf16_bits_to_f32(sb);
    double z = zeros ? 0.0 : 8.0;
    if (zeros && s != 0.0) z = fmin(fmax(__builtin_rint(-(double)lo / s), 0.0), 15.0);
    scales[i] = (uint16_t)sb;
    if (zeros) zeros[i] = (uint8_t)(int)z;
    for (int c = 0; c < n; c += 8) {
      load8<BF16>(x, base + c, v);
      uint32_t w = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double q = s == 0.0 ? z : fmin(fmax(__builtin_rint((double)v[j] / s) + z, 0.0), 15.0);
        w |= (uint32_t)(int)q << (j < 4 ? 8 * j : 8 * (j - 4) + 4);
      }
      *reinterpret_cast<uint32_t*>(codes + (base + c) / 2) = w;
    }
  }
}

// One thread per dword of 8 codes.
template <bool BF16>
__global__ __launch_bounds__(256) void int4_dequant_kernel(const uint8_t* __restrict__ codes,
                                                           const uint16_t* __restrict__ scales,
                                                           const uint8_t* __restrict__ zeros, int64_t rows, int64_t G,
                                                           int cols, int group, void* __restrict__ out) {
  const int64_t n8 = rows * (cols / 8);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / (cols / 8);
    const int64_t slot = r * G + (i % (cols / 8)) * 8 / group;
    const float s = bf16_bits_to_f32(scales[slot]);
    const int z = zeros ? zeros[slot] : 8;
    const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[i];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = s * (float)((int)((w >> (j < 4 ? 8 * j : 8 * (j - 4) + 4)) & 15u) - z);
      if (BF16)
        reinterpret_cast<uint16_t*>(out)[8 * i + j] = (uint16_t)f32_to_bf16_bits(v);
      else
        reinterpret_cast<float*>(out)[8 * i + j] = v;
    }
  }
}

static unsigned blocks_of(int64_t n) {
  const int64_t b = (n + 255) / 256;
  return (unsigned)(b < (1 << 20) ? b : (1 << 20));
}

hipError_t launch_int4_quantize(const void* x, bool bf16, int64_t rows, int64_t cols, int group, uint8_t* codes,
                                uint16_t* scales, uint8_t* zeros, hipStream_t stream) {
  const int64_t G = (cols + group - 1) / group, slots = rows * G;
  if (bf16)
    hipLaunchKernelGGL(int4_quantize_kernel<true>, dim3(blocks_of(slots)), dim3(256), 0, stream, x, slots, G, (int)cols,
                       group, codes, scales, zeros);
  else
    hipLaunchKernelGGL(int4_quantize_kernel<false>, dim3(blocks_of(slots)), dim3(256), 0, stream, x, slots, G,
                       (int)cols, group, codes, scales, zeros);
  return hipGetLastError();
}

hipError_t launch_int4_dequant(const Int4Weight& w, int64_t rows, int64_t cols, void* out, bool bf16_out,
                               hipStream_t stream) {
  const int64_t G = (cols + w.group - 1) / w.group, n8 = rows * (cols / 8);
  if (bf16_out)
    hipLaunchKernelGGL(int4_dequant_kernel<true>, dim3(blocks_of(n8)), dim3(256), 0, stream, w.codes, w.scales,
                       w.zeros, rows, G, (int)cols, w.group, out);
  else
    hipLaunchKernelGGL(int4_dequant_kernel<false>, dim3(blocks_of(n8)), dim3(256), 0, stream, w.codes, w.scales,
                       w.zeros, rows, G, (int)cols, w.group, out);
  return hipGetLastError();
}

}  // namespace nvfp4
