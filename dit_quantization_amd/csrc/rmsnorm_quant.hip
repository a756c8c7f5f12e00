// Residual addition, RMS norm and 8-bit output with scales (definition:
// include/int4.h, int4_rmsnorm_quant8).
#include "device_common.hpp"
#include "int4_kernels.hpp"

namespace nvfp4 {

// Nearest E4M3 byte to v (ties to even, saturating at 448), rounded once:
// the low half of the fp64 value becomes a sticky bit, which leaves 21
// significant bits that convert to fp32 exactly, and the converter rounds.
__device__ __forceinline__ float sticky_f32(double v) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t hi = (uint32_t)(b >> 32) | ((uint32_t)b != 0u ? 1u : 0u);
  return (float)__longlong_as_double((int64_t)((uint64_t)hi << 32));
}

__device__ __forceinline__ float norm_load(const void* p, int64_t i, bool bf16) {
  return bf16 ? bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}

// One workgroup per row; three passes over its elements.
__global__ __launch_bounds__(256) void rmsnorm_quant_kernel(NormArgs a) {
  __shared__ double red[256];
  const int t = threadIdx.x;
  const int step = a.group ? a.group : a.cols, G = (a.cols + step - 1) / step;
  const double top = a.e4m3 ? 448.0 : 127.0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    auto h_at = [&](int c) {
      const float x = norm_load(a.x, r * a.x_stride + c, a.x_bf16);
      if (!a.residual) return x;
      const float h = x + norm_load(a.residual, r * a.res_stride + c, a.res_bf16);
      return a.res_bf16 ? bf16_bits_to_f32(f32_to_bf16_bits(h)) : h;
    };
    auto y_at = [&](int c) { return (double)h_at(c) * (a.weight ? (double)norm_load(a.weight, c, a.w_bf16) : 1.0); };
    double ss = 0.0;
    for (int c = t; c < a.cols; c += 256) ss += (double)h_at(c) * (double)h_at(c);
    red[t] = ss;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
      if (t < o) red[t] += red[t + o];
      __syncthreads();
    }
    const double inv = 1.0 / sqrt(red[0] / a.cols + a.eps);
    __syncthreads();
    for (int g = 0; g < G; ++g) {
      const int c0 = g * step, c1 = min(c0 + step, a.cols);
      double m = 0.0;
      for (int c = c0 + t; c < c1; c += 256) m = fmax(m, fabs(y_at(c)));
      red[t] = m;
      __syncthreads();
      for (int o = 128; o > 0; o >>= 1) {
        if (t < o) red[t] = fmax(red[t], red[t + o]);
        __syncthreads();
      }
      m = red[0];
      __syncthreads();
      float s = m > 0.0 ? (float)(m * inv / top) : 0.0f;
      if (s == 0.0f) s = 1.0f;
      if (t == 0) a.scales[r * G + g] = s;
      const double k = m > 0.0 ? inv / (double)s : 0.0;
      for (int c = c0 + t; c < c1; c += 256) {
        const double v = y_at(c) * k;
        uint32_t q;
        if (a.e4m3) {
          const float f = fminf(fmaxf(sticky_f32(v), -448.0f), 448.0f);
          q = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f, f, 0, false) & 0xFFu;
        } else {
          q = (uint32_t)(int)fmin(fmax(__builtin_rint(v), -127.0), 127.0) & 0xFFu;
        }
        reinterpret_cast<uint8_t*>(a.codes)[r * a.cols + c] = (uint8_t)q;
      }
    }
    __syncthreads();
    if (a.residual)
      for (int c = t; c < a.cols; c += 256) {
        const float h = h_at(c);
        if (a.res_bf16)
          reinterpret_cast<uint16_t*>(a.residual_out)[r * a.cols + c] = (uint16_t)(__float_as_uint(h) >> 16);
        else
          reinterpret_cast<float*>(a.residual_out)[r * a.cols + c] = h;
      }
  }
}

hipError_t launch_rmsnorm_quant8(const NormArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.rows < (1 << 20) ? a.rows : (1 << 20)));
  hipLaunchKernelGGL(rmsnorm_quant_kernel, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace nvfp4
