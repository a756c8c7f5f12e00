// Weights to E4M3 with a scale for each 128 x 128 block, and activations (or
// SiLU(gate) x) to INT8 or E4M3 with a scale for each group of 32, 64 or 128
// columns (definitions: include/fp8.h).
//
// Both are one pass over memory: the values that share a scale stay in
// registers between the maximum and the codes.  Codes are decided by fp64
// quotients (the multiply-add runs at the fp32 rate here).
#include "device_common.hpp"
#include "encode8.hpp"
#include "fp8_kernels.hpp"
#include "lanes.hpp"

namespace nvfp4 {

// ---- weights.  A workgroup of 256 threads has one block: 16 lanes a row of
// 128 columns (8 each), 16 rows at a time, 8 vectors a thread, so that a block
// is read once.  14336 x 4096: fp32 51.4 us, 5.7 TB/s, bf16 33.8 us, 5.2 TB/s:
// memory.  About a block a CU (1100 x 4112, 7.7 us): the latency of one load and
// some 900 instructions behind it, which more threads a block hardly shorten
// (kernels alone, without the binding: 128, 256, 512 and 1024 threads 10.1, 7.7,
// 7.4 and 7.6 us; bf16 14336 x 4096 38.5, 33.8, 33.9 and 38.5).
template <bool BF>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(const void* __restrict__ x, int64_t stride, int64_t rows,
                                                           int cols, int blocks_k, uint8_t* __restrict__ codes,
                                                           float* __restrict__ scales) {
  constexpr int V = 8;
  const int bk = (int)(blockIdx.x % (unsigned)blocks_k);
  const int64_t bn = blockIdx.x / (unsigned)blocks_k;
  const int lane = threadIdx.x & 15, row0 = threadIdx.x >> 4;
  const int col = 128 * bk + 8 * lane;
  Vec8<BF> v[V];
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t r = 128 * bn + row0 + 16 * i;
    v[i].zero();
    if (r < rows && col < cols) v[i].load(x, r * stride + col);
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[i].at(j)));
  const auto most = [](float a, float b) { return fmaxf(a, b); };
  top = lanes_all<64>(top, most);
  __shared__ float part[4];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const float s = scale_for((double)top, 448.0);
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t r = 128 * bn + row0 + 16 * i;
    if (r < rows && col < cols) {
      double d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = (double)v[i].at(j);
      *reinterpret_cast<u32x2*>(codes + r * cols + col) = encode_quotients(d, s, true);
    }
  }
}

hipError_t launch_fp8_quantize(const void* x, bool bf16, int64_t stride, int64_t rows, int64_t cols, uint8_t* codes,
                               float* scales, hipStream_t stream) {
  const int blocks_k = (int)((cols + 127) / 128);
  // at most 2^22 workgroups a launch (a launch counts its threads in 32 bits), whole rows of blocks
  const int64_t step = 128 * (((int64_t)1 << 22) / blocks_k);
  for (int64_t r0 = 0; r0 < rows; r0 += step) {
    const int64_t n = rows - r0 < step ? rows - r0 : step;
    const void* xr = reinterpret_cast<const char*>(x) + r0 * stride * (bf16 ? 2 : 4);
    uint8_t* cr = codes + r0 * cols;
    float* sr = scales + r0 / 128 * blocks_k;
    const dim3 grid((unsigned)((n + 127) / 128 * blocks_k));
    if (bf16)
      hipLaunchKernelGGL(fp8_quantize_kernel<true>, grid, dim3(256), 0, stream, xr, stride, n, (int)cols, blocks_k, cr, sr);
    else
      hipLaunchKernelGGL(fp8_quantize_kernel<false>, grid, dim3(256), 0, stream, xr, stride, n, (int)cols, blocks_k, cr, sr);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---- activations.  A row is cut into slots of 16 columns, filled up to whole
// groups, and slots go to threads in order, so that a group is 2, 4 or 8
// neighbouring lanes.  4096 x 14336 bf16 to E4M3: 36 us, 4.9 TB/s; SiLU(gate) x
// 60 us, 4.9 TB/s: memory, and fp64 arithmetic (a table's read, a product and a
// quotient a value) that would take half as long alone.

// g / (1 + exp(-g)) to within 2^-45 of itself: exp(-g) = 2^n exp(r), |r| <= ln 2
// / 2, by 12 terms of its series (the rest is below 2^-47), and a reciprocal of
// the hardware's estimate (23 bits) and one Newton step.  g beyond 700 counts as
// 700 in the exponential: the product is below 10^-260, or g, either way.
__device__ __forceinline__ double silu64(float g) {
  constexpr double kMagic = 6755399441055744.0;  // 1.5 2^52: leaves the nearest integer in the low bits
  constexpr double kLog2e = 1.4426950408889634, kLn2 = 0.6931471805599453;
  const double z = (double)g, v = -(double)__builtin_amdgcn_fmed3f(g, -700.0f, 700.0f);
  const double m = __builtin_fma(v, kLog2e, kMagic);
  const double r = __builtin_fma(m - kMagic, -kLn2, v);
  double e = 1.0 / 39916800.0;
  constexpr double kInv[11] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320,
                               1.0 / 362880, 1.0 / 3628800};
#pragma unroll
  for (int i = 10; i >= 0; --i) e = __builtin_fma(e, r, kInv[i]);
  const double d = 1.0 + __builtin_amdgcn_ldexp(e, (int)__double_as_longlong(m));
  const double q = __builtin_amdgcn_rcp(d);
  return z * __builtin_fma(q, __builtin_fma(-d, q, 1.0), q);
}

// The same of a bf16 gate from a table: of both signs and all magnitudes from
// 2^-16 up to 2^8, computed when this file is compiled (within 2^-48: ln 2 in two
// parts, 17 terms of the series).  Below it g / 2 + g^2 / 4 is within 2^-52, above
// it g is, and under -2^8 a product with any x is below fp32's range.
constexpr uint32_t kTableFirst = (127 - 16) << 7, kTableSize = 24 << 7;
constexpr uint32_t kTableStride = kTableSize + 2;  // in LDS: behind the entries of a sign, that of a 0
struct SiluTable {
  double v[2 * kTableSize];
  constexpr SiluTable() : v() {
    constexpr double kLn2High = 0x1.62e42fefap-1, kLn2Low = 0x1.cf79abc9e3b3ap-40;  // 38 bits, and the rest
    for (uint32_t i = 0; i < kTableSize; ++i) {
      const double g = (double)__builtin_bit_cast(float, (kTableFirst + i) << 16);
      const int n = (int)(g * 1.4426950408889634 + 0.5);
      const double r = (n * kLn2High - g) + n * kLn2Low;  // exp(-g) = 2^-n exp(r), |r| <= ln 2 / 2
      double e = 1.0;
      for (int k = 17; k > 0; --k) e = 1.0 + e * r / k;
      e *= __builtin_bit_cast(double, (uint64_t)(1023 - n) << 52);
      v[i] = g / (1.0 + e);
      v[kTableSize + i] = -g * e / (1.0 + e);
    }
  }
};
__device__ constexpr SiluTable kSilu{};
__device__ __forceinline__ void fill_table(double* table) {
  static_assert(kTableSize % 512 == 0, "two entries a thread at a time");
#pragma unroll
  for (uint32_t i = 0; i < 2 * kTableSize; i += 2 * 512) {
    const uint32_t at = i + 2 * threadIdx.x;
    *reinterpret_cast<u32x4*>(table + at + (at >= kTableSize ? kTableStride - kTableSize : 0)) =
        *reinterpret_cast<const u32x4*>(kSilu.v + at);
  }
  if (threadIdx.x < 2) table[kTableSize + threadIdx.x * kTableStride] = threadIdx.x ? -0.0 : 0.0;
  __syncthreads();
}

// f over the L = 2, 4 or 8 lanes of a group.
template <class T, class F>
__device__ __forceinline__ T group_all(T v, int L, F f) {
  v = f(v, dpp<kDppXor1>(v));
  if (L >= 4) v = f(v, dpp<kDppXor2>(v));
  if (L >= 8) v = f(v, dpp<kDppHalfMirror>(v));
  return v;
}

// TABLE (bf16 gates): a grid of as many workgroups as fit at once, each with a
// copy of the table in LDS.  For 2 million values and more: an exponential is 24
// of 47 vector instructions a value (4096 x 14336 60 against 88 us, 512 x 14336 10.8
// against 12.3, 128 x 14336 4.9 against 5.0).  Gates of 0 are an entry of it; others
// outside take some 15 instructions each, in the lanes that have them (gates of spread 2, 0.02, 0, 2000:
// 60, 64, 60, 75 us; one after the other, read again, with an exponential: 67, 137, 238, 240).
template <bool BF, bool SILU, bool TABLE>
__global__ __launch_bounds__(TABLE ? 512 : 256) void fp8_quantize_act_kernel(ActArgs a, uint32_t slots, uint32_t per,
                                                                              uint32_t all, double q, double inv_q) {
  __shared__ __attribute__((aligned(16))) double table[TABLE ? 2 * kTableStride : 1];
  if (TABLE) fill_table(table);
  const int L = a.group / 16;
  // (rounds of whole workgroups, so that all lanes of a group are there)
  for (uint32_t first = blockIdx.x * blockDim.x; first < all; first += gridDim.x * blockDim.x) {
    // at / slots, per = 2^32 / slots rounded down: the first quotient is exact or one short
    const uint32_t at = first + threadIdx.x;
    uint32_t row = __umulhi(at, per), i = at - row * slots;
    if (i >= slots) {
      ++row;
      i -= slots;
    }
    const int64_t r = row;
    const int c = 16 * (int)i;
    const bool live = r < a.rows && c < a.cols;
    Vec8<BF> x[2], g[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x[h].zero();
      g[h].zero();
      if (live) {
        x[h].load(a.x, r * a.x_stride + c + 8 * h);
        if (SILU) g[h].load(a.gate, r * a.gate_stride + c + 8 * h);
      }
    }
    double y[16], top = 0.0;
    bool outside = false;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      y[j] = (double)x[j / 8].at(j % 8);
      if (SILU && !TABLE) y[j] *= silu64(g[j / 8].at(j % 8));
      if (TABLE) {
        const uint32_t w = g[j / 8].a[0][j % 8 / 2], bits = j & 1 ? w >> 16 : w & 0xFFFFu;
        const uint32_t entry = (bits & 0x7FFFu) - kTableFirst;
        outside |= entry >= kTableSize && entry != 0u - kTableFirst;  // (not a gate of 0)
        y[j] *= table[min(entry, kTableSize) + (bits >> 15) * kTableStride];
      }
    }
    if (TABLE && outside) {  // a lane with a gate beyond the table's range, few of them
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        // (from the vectors as they came: kept as fp64 they would take the registers of a workgroup a CU)
        const uint32_t xw = fresh(x[j / 8].a[0][j % 8 / 2]), gw = fresh(g[j / 8].a[0][j % 8 / 2]);
        const float f = __uint_as_float(j & 1 ? gw & 0xFFFF0000u : gw << 16);
        if (fabsf(f) < 0x1p-16f || fabsf(f) >= 0x1p8f) {
          const double gate = (double)f, of = (double)__uint_as_float(j & 1 ? xw & 0xFFFF0000u : xw << 16);
          const double half = fabsf(f) < 1.0f ? __builtin_fma(gate, 0.25, 0.5) : f > 0.0f ? 1.0 : 0.0;
          y[j] = of * (gate * half);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) top = fmax(top, fabs(y[j]));
    top = group_all(top, L, [](double p, double t) { return p > t ? p : t; });
    float s = (float)quotient(top, q, inv_q);
    s = s == 0.0f ? 1.0f : s;
    if (live) {
      u32x2 code[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (SILU || a.e4m3) code[h] = encode_quotients(y + 8 * h, s, a.e4m3);
        else code[h] = encode(x[h], s, false);
      }
      *reinterpret_cast<u32x4*>(reinterpret_cast<uint8_t*>(a.codes) + r * a.cols + c) =
          u32x4{code[0].x, code[0].y, code[1].x, code[1].y};
      if ((i & (L - 1)) == 0) a.scales[r * (int64_t)(slots / L) + i / L] = s;
    }
  }
}

hipError_t launch_fp8_quantize_act(const ActArgs& all, hipStream_t stream) {
  const int L = all.group / 16;
  const uint32_t slots = (uint32_t)((all.cols + all.group - 1) / all.group * L);  // >= 2
  const uint32_t per = (uint32_t)(((uint64_t)1 << 32) / slots);
  // at most 2^31 slots a launch, whole rows
  const int64_t step = ((int64_t)1 << 31) / slots;
  for (int64_t r0 = 0; r0 < all.rows; r0 += step) {
    ActArgs a = all;
    const int size = a.bf16 ? 2 : 4;
    a.rows = all.rows - r0 < step ? all.rows - r0 : step;
    a.x = reinterpret_cast<const char*>(all.x) + r0 * all.x_stride * size;
    if (a.gate) a.gate = reinterpret_cast<const char*>(all.gate) + r0 * all.gate_stride * size;
    a.codes = reinterpret_cast<char*>(all.codes) + r0 * all.cols;
    a.scales = all.scales + r0 * (slots / L);
    const uint32_t n = (uint32_t)(a.rows * slots);
    const double q = a.e4m3 ? 448.0 : 127.0;
#define ACT_CASE(BF, SILU, TABLE, GRID)                                                                        \
  hipLaunchKernelGGL((fp8_quantize_act_kernel<BF, SILU, TABLE>), dim3(GRID), dim3(TABLE ? 512 : 256), 0, stream, a, \
                     slots, per, n, q, 1.0 / q)
    if (a.gate && a.bf16 && n >= (1u << 17)) ACT_CASE(true, true, true, 768);
    else if (a.gate && a.bf16) ACT_CASE(true, true, false, (n + 255) / 256);
    else if (a.gate) ACT_CASE(false, true, false, (n + 255) / 256);
    else if (a.bf16) ACT_CASE(true, false, false, (n + 255) / 256);
    else ACT_CASE(false, false, false, (n + 255) / 256);
#undef ACT_CASE
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace nvfp4
