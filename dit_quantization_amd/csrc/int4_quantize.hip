// Group-scaled 4-bit integer weights (format: include/int4.h): the quantizer
// and its inverse.  Both stream, bound by memory.  In the quantizer a lane holds
// a vector of 8 consecutive elements (one dword of codes) and a group of 32,
// 64 or 128 is 4, 8 or 16 neighbouring lanes, so its range is a few lane
// exchanges.  A wave takes runs of 64 vectors of one row; where rows end on a
// group (the usual case) the whole tensor is one such row.  14336 x 4096: fp32
// quantize 266 MB in 47 us (5.7 TB/s), bf16 148 MB in 30.4 (4.9); dequant to
// bf16 148 MB in 23 us with the codes in the last-level cache, 32 without (4.6).
#include "device_common.hpp"
#include "int4_kernels.hpp"
#include "lanes.hpp"

namespace nvfp4 {

// Runs of 64 vectors that a wave keeps in flight, from a sweep over 1, 2, 4
// and 8 (us, weights read again after 3 others / after 14): quantize 14336 x
// 4096 fp32 46.9 / 46.8 with 1, 48.6 / 48.4 with 2; bf16 30.3 / 30.7 with 2, 35.4
// / 35.5 with 1; dequant to bf16 22.4 / 31.0 with 2, 24.8 / 36.8 with 1; to fp32
// 37.4 / 54.4 and 42.6 / 65.6.  4 runs gain nothing on large weights and lose on
// small ones.  (Inputs read non-temporally: fp32 49.6, bf16 30.5 and at 4096 x
// 4096 11.6 instead of 10.6, dequant 31.4.)
constexpr int runs_in_flight(bool quantize, bool bf16) { return quantize && !bf16 ? 1 : 2; }

// The rows a launch sees: the tensor's own, or one of all its elements.
struct RowView {
  int64_t rows, nv, padded;  // vectors of a row, and that rounded up to whole groups
  int64_t units;             // as many runs of a row as a wave keeps in flight, each
};

// per: elements of a vector
static RowView row_view(int64_t rows, int64_t cols, int group, int per, int runs) {
  RowView v;
  const bool flat = cols % group == 0;
  v.rows = flat ? 1 : rows;
  v.nv = (flat ? rows * cols : cols) / per;
  v.padded = (v.nv + group / per - 1) / (group / per) * (group / per);
  v.units = ((v.padded + 63) / 64 + runs - 1) / runs;
  return v;
}

template <bool BF16>
struct Raw {
  u32x4 a[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* x, int64_t vec) {
    const u32x4* p = reinterpret_cast<const u32x4*>(x) + (BF16 ? vec : 2 * vec);
    a[0] = p[0];
    if (!BF16) a[BF16 ? 0 : 1] = p[1];
  }
  __device__ __forceinline__ void zero() {
    a[0] = u32x4{0, 0, 0, 0};
    a[BF16 ? 0 : 1] = u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ float at(int j) const {
    if (BF16) return __uint_as_float(j & 1 ? a[0][j / 2] & 0xFFFF0000u : a[0][j / 2] << 16);
    return __uint_as_float(a[BF16 ? 0 : j / 4][j % 4]);
  }
};

// rne(w / s) for |w / s| < 16 and s >= 2^-100 (8 significant bits), with inv
// the hardware's estimate of 1 / s.
//  * bf16 w: a quotient of two 8-bit numbers is half way between integers or
//    further from it than 2^-13, and one corrected step gives it to within an
//    ulp, exactly where it has few bits, as half way does.
//  * fp32 w: t = w inv is off by less than 2^-18; only where that may decide
//    is w compared with the border itself, (k + 1/2) s for k = floor(t), which
//    has 13 bits and is exact (a floor that is one too low next to an integer
//    does not matter).
__device__ __forceinline__ float quotient_bf16(float w, float s, float inv) {
  const float q = w * inv;
  return __builtin_fmaf(__builtin_fmaf(-q, s, w), inv, q);
}
constexpr float kHalfway = 0.4999f;

__device__ __forceinline__ float nearest_f32(float w, float s, float t) {
  const float k = __builtin_floorf(t), border = (k + 0.5f) * s;
  const float even = __builtin_rintf(k + 0.5f);
  const float down = w < border ? k : even;
  return w > border ? k + 1.0f : down;
}

template <bool BF16, int RUNS>
__global__ __launch_bounds__(256) void int4_quantize_kernel(const void* __restrict__ x, RowView rv, int shift,
                                                            int64_t G, uint8_t* __restrict__ codes,
                                                            uint16_t* __restrict__ scales,
                                                            uint8_t* __restrict__ zeros) {
  const int lane = threadIdx.x & 63, L = 1 << shift;  // vectors of a group
  const int64_t n_units = rv.rows * rv.units;
  for (int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < n_units;
       u += (int64_t)gridDim.x * 4) {
    const int64_t row = rv.rows == 1 ? 0 : u / rv.units;
    const int64_t v0 = (u - row * rv.units) * RUNS * 64 + lane;
    Raw<BF16> raw[RUNS];
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      if (v0 + 64 * k < rv.nv) raw[k].load(x, row * rv.nv + v0 + 64 * k);
      else raw[k].zero();
    }
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      const int64_t v = v0 + 64 * k;
      float lo = 0.0f, hi = 0.0f, w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = raw[k].at(j);
        lo = fminf(lo, w[j]);
        hi = fmaxf(hi, w[j]);
      }
      lo = lanes_all(lo, L, [](float p, float q) { return fminf(p, q); });
      hi = lanes_all(hi, L, [](float p, float q) { return fmaxf(p, q); });
      const double range = zeros ? ((double)hi - (double)lo) * (1.0 / 15.0) : (double)fmaxf(hi, -lo) * (1.0 / 7.0);
      const uint32_t sb = f32_to_bf16_bits((float)range);
      const float s = bf16_bits_to_f32(sb);
      const float inv = __builtin_amdgcn_rcpf(s);
      const bool odd_scale = s < 0x1p-100f;  // also 0
      float t[9];                            // the eight codes before the zero point, and that
      if constexpr (BF16) {
#pragma unroll
        for (int j = 0; j < 9; ++j) t[j] = __builtin_rintf(quotient_bf16(j < 8 ? w[j] : -lo, s, inv));
      } else {
        bool near = false;
#pragma unroll
        for (int j = 0; j < 9; ++j) {
          const float q = (j < 8 ? w[j] : -lo) * inv;
          t[j] = __builtin_rintf(q);
          near |= fabsf(q - t[j]) > kHalfway;
        }
        if (near) {
#pragma unroll
          for (int j = 0; j < 9; ++j) {
            const float v = j < 8 ? w[j] : -lo;
            t[j] = nearest_f32(v, s, v * inv);
          }
        }
      }
      if (odd_scale) {
        // fp64: w has 24 significant bits and s 8, so a quotient that is not
        // half way is further from it than fp64 rounds
#pragma unroll
        for (int j = 0; j < 9; ++j)
          t[j] = s == 0.0f ? 0.0f : (float)__builtin_rint((double)(j < 8 ? w[j] : -lo) / (double)s);
      }
      const float z = zeros ? __builtin_amdgcn_fmed3f(t[8], 0.0f, 15.0f) : 8.0f;
      uint32_t word = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float c0 = __builtin_amdgcn_fmed3f(t[b] + z, 0.0f, 15.0f);
        const float c1 = __builtin_amdgcn_fmed3f(t[4 + b] + z, 0.0f, 15.0f);
        word |= (uint32_t)__builtin_fmaf(c1, 16.0f, c0) << (8 * b);
      }
      if (v < rv.nv) {
        reinterpret_cast<uint32_t*>(codes)[row * rv.nv + v] = word;
        if ((lane & (L - 1)) == 0) {
          const int64_t slot = row * G + (v >> shift);
          scales[slot] = (uint16_t)sb;
          if (zeros) zeros[slot] = (uint8_t)(uint32_t)z;
        }
      }
    }
  }
}

// A lane makes 16 bytes: 8 bf16 values of a dword of codes, or the 4 fp32
// values of its low or its high nibbles (then two lanes read one dword).
template <bool BF16, int RUNS>
__global__ __launch_bounds__(256) void int4_dequant_kernel(const uint8_t* __restrict__ codes,
                                                           const uint16_t* __restrict__ scales,
                                                           const uint8_t* __restrict__ zeros, RowView rv, int shift,
                                                           int64_t G, void* __restrict__ out) {
  constexpr int HALVES = BF16 ? 1 : 2;
  const int lane = threadIdx.x & 63;
  const int64_t n_units = rv.rows * rv.units;
  for (int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < n_units;
       u += (int64_t)gridDim.x * 4) {
    const int64_t row = rv.rows == 1 ? 0 : u / rv.units;
    const int64_t v0 = (u - row * rv.units) * RUNS * 64 + lane;
    uint32_t w[RUNS], sb[RUNS], z[RUNS];
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      const int64_t v = min(v0 + 64 * k, rv.nv - 1);
      const int64_t slot = row * G + (v >> shift);
      w[k] = reinterpret_cast<const uint32_t*>(codes)[(row * rv.nv + v) / HALVES];
      sb[k] = scales[slot];
      z[k] = zeros ? zeros[slot] : 8u;
    }
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      const int64_t v = v0 + 64 * k;
      const float s = bf16_bits_to_f32(sb[k]), zf = (float)z[k];
      const uint32_t half[2] = {(BF16 || (lane & 1) == 0 ? w[k] : w[k] >> 4) & 0x0F0F0F0Fu, (w[k] >> 4) & 0x0F0F0F0Fu};
      float f[8 / HALVES];
#pragma unroll
      for (int j = 0; j < 8 / HALVES; ++j) f[j] = s * ((float)((half[j / 4] >> (8 * (j & 3))) & 0xFFu) - zf);
      if (v >= rv.nv) continue;
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = BF16 ? pk_bf16(f[BF16 ? 2 * j : 0], f[BF16 ? 2 * j + 1 : 0]) : __float_as_uint(f[j]);
      __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(out) + row * rv.nv + v);
    }
  }
}

static dim3 stream_grid(const RowView& v) {
  const int64_t b = (v.rows * v.units + 3) / 4;
  return dim3((unsigned)(b < (1 << 20) ? b : (1 << 20)));
}

hipError_t launch_int4_quantize(const void* x, bool bf16, int64_t rows, int64_t cols, int group, uint8_t* codes,
                                uint16_t* scales, uint8_t* zeros, hipStream_t stream) {
  const RowView v = row_view(rows, cols, group, 8, runs_in_flight(true, bf16));
  const int64_t G = (cols + group - 1) / group;
#define INT4_QUANTIZE(B)                                                                                        \
  hipLaunchKernelGGL((int4_quantize_kernel<B, runs_in_flight(true, B)>), stream_grid(v), dim3(256), 0, stream, x, \
                     v, __builtin_ctz(group / 8), G, codes, scales, zeros)
  if (bf16) INT4_QUANTIZE(true);
  else INT4_QUANTIZE(false);
#undef INT4_QUANTIZE
  return hipGetLastError();
}

hipError_t launch_int4_dequant(const Int4Weight& w, int64_t rows, int64_t cols, void* out, bool bf16_out,
                               hipStream_t stream) {
  const RowView v = row_view(rows, cols, w.group, bf16_out ? 8 : 4, runs_in_flight(false, bf16_out));
  const int64_t G = (cols + w.group - 1) / w.group;
#define INT4_DEQUANT(B)                                                                                            \
  hipLaunchKernelGGL((int4_dequant_kernel<B, runs_in_flight(false, B)>), stream_grid(v), dim3(256), 0, stream,     \
                     w.codes, w.scales, w.zeros, v, __builtin_ctz(w.group / (B ? 8 : 4)), G, out)
  if (bf16_out) INT4_DEQUANT(true);
  else INT4_DEQUANT(false);
#undef INT4_DEQUANT
  return hipGetLastError();
}

}  // namespace nvfp4
