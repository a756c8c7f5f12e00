// Decode products y = x W^T for group-scaled 4-bit integer weights and bf16,
// INT8 or E4M3 activations, M <= 16 rows (format: include/int4.h).
#include "device_common.hpp"
#include "int4_kernels.hpp"

namespace nvfp4 {

template <Act A>
__device__ __forceinline__ float act_value(const void* x, int64_t i) {
  if (A == Act::kBf16) return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(x)[i]);
  if (A == Act::kI8) return (float)reinterpret_cast<const int8_t*>(x)[i];
  const uint32_t b = reinterpret_cast<const uint8_t*>(x)[i];
  const float v = e4m3_to_f32(b & 0x7Fu);
  return b & 0x80u ? -v : v;
}

// One wave per output element; the lanes take the dwords of 8 codes in turn.
template <Act A>
__global__ __launch_bounds__(256) void int4_gemv_kernel(Int4Act x, Int4Weight w, int M, int64_t N, int K, int G,
                                                        void* __restrict__ y, int bf16_out) {
  const int lane = threadIdx.x & 63;
  for (int64_t o = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); o < M * N; o += (int64_t)gridDim.x * 4) {
    const int m = (int)(o / N);
    const int64_t n = o % N;
    float acc = 0.0f;
    for (int d = lane; d < K / 8; d += 64) {
      const int64_t slot = 8 * d / w.group;
      const uint32_t c = *reinterpret_cast<const uint32_t*>(w.codes + n * (K / 2) + 4 * (int64_t)d);
      const int z = w.zeros ? w.zeros[n * G + slot] : 8;
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        dot = __builtin_fmaf(act_value<A>(x.x, (int64_t)m * K + 8 * d + j),
                             (float)((int)((c >> (j < 4 ? 8 * j : 8 * (j - 4) + 4)) & 15u) - z), dot);
      const float s = bf16_bits_to_f32(w.scales[n * G + slot]);
      acc = __builtin_fmaf(dot, x.grouped ? s * x.scales[m * G + slot] : s, acc);
    }
#pragma unroll
    for (int i = 32; i > 0; i >>= 1) acc += __shfl_xor(acc, i);
    if (A != Act::kBf16 && !x.grouped) acc *= x.scales[m];
    if (lane == 0) {
      if (bf16_out)
        reinterpret_cast<uint16_t*>(y)[o] = (uint16_t)f32_to_bf16_bits(acc);
      else
        reinterpret_cast<float*>(y)[o] = acc;
    }
  }
}

hipError_t launch_int4_gemv(const Int4Act& x, const Int4Weight& w, int64_t M, int64_t N, int64_t K, void* y,
                            bool bf16_out, hipStream_t stream) {
  const int64_t b = (M * N + 3) / 4;
  const dim3 grid((unsigned)(b < (1 << 20) ? b : (1 << 20)));
  const int G = (int)((K + w.group - 1) / w.group);
#define INT4_GEMV(A) \
  hipLaunchKernelGGL(int4_gemv_kernel<A>, grid, dim3(256), 0, stream, x, w, (int)M, N, (int)K, G, y, bf16_out ? 1 : 0)
  if (x.type == Act::kBf16) INT4_GEMV(Act::kBf16);
  else if (x.type == Act::kI8) INT4_GEMV(Act::kI8);
  else INT4_GEMV(Act::kE4m3);
#undef INT4_GEMV
  return hipGetLastError();
}

}  // namespace nvfp4
