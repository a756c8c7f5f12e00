// Vectors of 8 columns and their encoding as INT8 or E4M3, shared by the
// kernels that quantize to 8 bits.
#pragma once
#include "device_common.hpp"
#include "lanes.hpp"

namespace nvfp4 {

// The value with its low 32 bits folded into a sticky bit: 21 significant
// bits, which convert to fp32 exactly, so that a later rounding to 8 bits is
// the only one.
__device__ __forceinline__ float sticky_f32(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t hi = (uint32_t)(b >> 32) | min((uint32_t)b, 1u);
  return (float)__longlong_as_double((int64_t)((uint64_t)hi << 32));
}

// 1 / x for positive normal x: the hardware estimate and two Newton steps (each
// squares the error).
__device__ __forceinline__ double rcp64(double x) {
  double y = __builtin_amdgcn_rcp(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __builtin_fma(y, __builtin_fma(-x, y, 1.0), y);
  return y;
}

// 8 columns as they lie in memory, bf16 or fp32.
template <bool BF16>
struct Vec8 {
  u32x4 a[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const u32x4* q = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(p) + i * (BF16 ? 2 : 4));
    a[0] = q[0];
    if (!BF16) a[BF16 ? 0 : 1] = q[1];
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    u32x4* q = reinterpret_cast<u32x4*>(reinterpret_cast<char*>(p) + i * (BF16 ? 2 : 4));
    q[0] = a[0];
    if (!BF16) q[1] = a[BF16 ? 0 : 1];
  }
  __device__ __forceinline__ void zero() {
    a[0] = u32x4{0, 0, 0, 0};
    a[BF16 ? 0 : 1] = u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ float at(int j) const {
    if (BF16) return __uint_as_float(j & 1 ? a[0][j / 2] & 0xFFFF0000u : a[0][j / 2] << 16);
    return __uint_as_float(a[BF16 ? 0 : j / 4][j % 4]);
  }
  __device__ __forceinline__ void set(const float v[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!BF16) a[BF16 ? 0 : j / 4][j % 4] = __float_as_uint(v[j]);
      else if (j & 1) a[0][j / 2] = pk_bf16(v[j - 1], v[j]);
    }
  }
};

// 8 codes of y / s = p k as two dwords.
__device__ __forceinline__ u32x2 encode_i8(const double p[8], double k) {
  u32x2 q;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // adding 1.5 2^52 rounds to the nearest integer, ties to even, and
      // leaves it in the low bits
      const double r = __builtin_fma(p[4 * d + j], k, 6755399441055744.0);
      const int c = min(max((int)__double_as_longlong(r), -127), 127);
      w |= ((uint32_t)c & 0xFFu) << (8 * j);
    }
    q[d] = w;
  }
  return q;
}
__device__ __forceinline__ u32x2 encode_e4m3(const double p[8], double k) {
  u32x2 q;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __builtin_amdgcn_fmed3f(sticky_f32(p[4 * d + j] * k), -448.0f, 448.0f);
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    q[d] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
  }
  return q;
}

// INT8 codes from exact fp32 products p and k rounded to fp32: u = p k is off
// by less than 2^-22 |u| < 2^-15; `near` where that may decide a code.  (For
// E4M3 the test for half way costs more than it saves.)
__device__ __forceinline__ u32x2 encode_i8_fast(const float p[8], float k, bool& near) {
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float u = p[j] * k;
    const float m = u + 12582912.0f;  // 1.5 2^23: the low byte is the code
    near |= fabsf(u - (m - 12582912.0f)) > 0.49996f;
    b[j] = __float_as_uint(m);
  }
  u32x2 q;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * d + 1], b[4 * d], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * d + 3], b[4 * d + 2], 0x04000c0cu);
    q[d] = lo | hi;
  }
  return q;
}
// A value the compiler takes for a new one, so that what is computed from it
// is not kept from earlier.
template <class T>
__device__ __forceinline__ T fresh(T v) {
  asm volatile("" : "+v"(v));
  return v;
}

// v / s, correctly rounded where the quotient has few bits, so that ties are
// decided as such: k is 1 / s to within an ulp or two, and the remainder of the
// first estimate is exact there.
__device__ __forceinline__ double quotient(double v, double s, double k) {
  const double q = v * k;
  return __builtin_fma(__builtin_fma(-q, s, v), k, q);
}

// 8 codes of v / s, decided by the exact quotients.
__device__ __forceinline__ u32x2 encode_quotients(const double v[8], float s, bool e4m3) {
  const double d = (double)s, k = rcp64(d);
  double q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = quotient(v[j], d, k);
  return e4m3 ? encode_e4m3(q, 1.0) : encode_i8(q, 1.0);
}

// 8 codes of exact fp32 or bf16 values v / s.  INT8 in fp32 unless a quotient is
// next to half way between two codes (or the scale is next to the end of fp32's
// range).
template <bool BF16>
__device__ __forceinline__ u32x2 encode(const Vec8<BF16>& v, float s, bool e4m3) {
  bool exact = e4m3 || s < 0x1p-120f;
  u32x2 q;
  if (!e4m3) {
    float p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = v.at(j);
    q = encode_i8_fast(p, (float)rcp64((double)s), exact);
  }
  if (exact) {
    double d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = (double)fresh(v.at(j));
    q = encode_quotients(d, s, e4m3);
  }
  return q;
}

// fp32(top / Q), 1 where that is 0.
__device__ __forceinline__ float scale_for(double top, double q) {
  const float s = (float)(top / q);
  return s == 0.0f ? 1.0f : s;
}

}  // namespace nvfp4
