// Block-scaled FP8 product y = x^ W^^T (definition: include/fp8.h):
//   y[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_{k in b} x[m, k] w[n, k]
// with b the blocks of 128 columns.
#include "device_common.hpp"
#include "fp8_kernels.hpp"
#include "lanes.hpp"

namespace nvfp4 {

// Four E4M3 values (a dword) as bf16, exact.
__device__ __forceinline__ u32x2 widen4(uint32_t w) {
  return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))};
}
// Half a 16-byte chunk (8 values) as an operand of the bf16 matrix instruction.
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi) {
  const u32x2 a = widen4(lo), b = widen4(hi);
  return __builtin_bit_cast(bf16x8, u32x4{a.x, a.y, b.x, b.y});
}

// acc += xs ws d.  The product of the scales is used where it is a normal number
// in all lanes; elsewhere it could leave fp32's range although xs ws d does not.
__device__ __forceinline__ void add_scaled(f32x4 d, float ws, float xs, f32x4& acc) {
  constexpr int kNotNormal = 0x003 | 0x004 | 0x200 | 0x010 | 0x080 | 0x020 | 0x040;  // NaN, infinity, subnormal, zero
  const float s = ws * xs;
  if (__ballot(__builtin_amdgcn_classf(s, kNotNormal)) == 0) {
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(d[r], s, acc[r]);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] += (float)((double)d[r] * ((double)ws * (double)xs));
  }
}

// ---- few rows.  A workgroup of W waves has 16 MT rows of x and 16 NT rows of
// the weight; its waves take the blocks of 128 columns in turn, straight from
// memory into registers, P blocks ahead, and their sums meet in LDS.  Values
// are widened to bf16, whose products and sums are fp32's (the FP8 matrix
// instruction aligns the products of 8 columns to the largest and cuts them
// off 13 bits below it); memory and not the instruction bounds these calls.
// Lane l of a 16 x 16 tile feeds row l % 16 and the columns 16 (l / 16) .. + 15
// and 64 more of a block, the same ones of both operands.  Loads past a row's
// end or of rows that are not there return zeros.
template <int MT, int NT, int W, int P>
__global__ __launch_bounds__(64 * W) void fp8_gemm_rows_kernel(Fp8Product p) {
  constexpr int BM = 16 * MT, BN = 16 * NT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int tiles_n = (p.N + BN - 1) / BN;
  const int n0 = (int)(blockIdx.x % (unsigned)tiles_n) * BN;
  const int64_t m0 = (int64_t)(blockIdx.x / (unsigned)tiles_n) * BM;
  const int rows = (int)min((int64_t)BM, p.M - m0);
  const int G = (p.K + 127) / 128;
  const __amdgpu_buffer_rsrc_t wbuf =
      make_buf(p.w + (int64_t)n0 * p.K, (uint32_t)min(BN, p.N - n0) * (uint32_t)p.K);
  const __amdgpu_buffer_rsrc_t xbuf =
      make_buf(p.x + m0 * p.K, (uint32_t)rows * (uint32_t)p.K);
  const __amdgpu_buffer_rsrc_t sbuf =
      make_buf(p.xs + m0 * G, (uint32_t)rows * (uint32_t)G * 4u);
  const float* ws = p.ws + (int64_t)(n0 / 128) * G;
  uint32_t w_off[NT], x_off[MT], s_off[MT];
#pragma unroll
  for (int t = 0; t < NT; ++t) w_off[t] = (uint32_t)(16 * t + l16) * (uint32_t)p.K;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    x_off[t] = (uint32_t)(16 * t + l16) * (uint32_t)p.K;
    s_off[t] = (uint32_t)min(16 * t + l16, rows - 1) * (uint32_t)G * 4u;
  }
  u32x4 wq[P][NT][2], xq[P][MT][2];
  float xs[P][MT], wsc[P];
  const auto load = [&](int s, int b) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t k = 128u * (uint32_t)b + 64u * h + 16u * (uint32_t)g;
      const bool ok = k < (uint32_t)p.K;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        wq[s][t][h] = __builtin_amdgcn_raw_buffer_load_b128(wbuf, ok ? w_off[t] + k : kBufOOB, 0, 0);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        xq[s][t][h] = __builtin_amdgcn_raw_buffer_load_b128(xbuf, ok ? x_off[t] + k : kBufOOB, 0, 0);
    }
    const int bs = min(b, G - 1);  // a block past the end adds zeros
#pragma unroll
    for (int t = 0; t < MT; ++t)
      xs[s][t] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sbuf, s_off[t] + 4u * (uint32_t)bs, 0, 0));
    wsc[s] = ws[bs];
  };
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < P; ++s) load(s, wave + W * s);
  for (int b = wave; b < G; b += W * P) {
#pragma unroll
    for (int s = 0; s < P; ++s) {
      bf16x8 xb[MT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 4; ++h) xb[i][h] = widen8(xq[s][i][h / 2][2 * (h & 1)], xq[s][i][h / 2][2 * (h & 1) + 1]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        bf16x8 wb[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) wb[h] = widen8(wq[s][t][h / 2][2 * (h & 1)], wq[s][t][h / 2][2 * (h & 1) + 1]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          f32x4 d = {0, 0, 0, 0};
#pragma unroll
          for (int h = 0; h < 4; ++h) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[h], xb[i][h], d, 0, 0, 0);
          add_scaled(d, wsc[s], xs[s][i], acc[i][t]);
        }
      }
      load(s, b + W * (s + P));
    }
  }
  // the waves' sums, in wave order
  __shared__ f32x4 part[W > 1 ? W : 1][MT * NT][64];
  if (W > 1) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) part[wave][i * NT + t][lane] = acc[i][t];
    __syncthreads();
  }
  // a wave finishes the tiles wave, wave + W, ...
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if ((i * NT + t) % W != wave) continue;
      f32x4 v = acc[i][t];
      if (W > 1) {
        v = part[0][i * NT + t][lane];
#pragma unroll
        for (int u = 1; u < W; ++u) v += part[u][i * NT + t][lane];
      }
      // lane: row m of x, four rows n of the weight
      const int m = 16 * i + l16, n = n0 + 16 * t + 4 * g;
      if (m >= rows) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (n + r >= p.N) break;
        const int64_t at = (m0 + m) * p.N + n + r;
        if (p.bf16) reinterpret_cast<uint16_t*>(p.y)[at] = (uint16_t)f32_to_bf16_bits(v[r]);
        else reinterpret_cast<float*>(p.y)[at] = v[r];
      }
    }
}

// Launches of a kernel with tiles of bm rows of x and bn of the weight: as many
// rows of x at once as 2^22 workgroups take.
template <class F>
hipError_t launch_tiles(const Fp8Product& all, int bm, int bn, F launch) {
  const int64_t tiles_n = (all.N + bn - 1) / bn;
  const int64_t step = (((int64_t)1 << 22) / tiles_n) * bm;
  for (int64_t m0 = 0; m0 < all.M; m0 += step) {
    Fp8Product p = all;
    p.M = all.M - m0 < step ? all.M - m0 : step;
    p.x += m0 * all.K;
    p.xs += m0 * ((all.K + 127) / 128);
    p.y = reinterpret_cast<char*>(all.y) + m0 * all.N * (all.bf16 ? 2 : 4);
    launch(p, dim3((unsigned)((p.M + bm - 1) / bm * tiles_n)));
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int MT, int NT, int W, int P>
hipError_t launch_rows(const Fp8Product& p, hipStream_t stream) {
  return launch_tiles(p, 16 * MT, 16 * NT, [=](const Fp8Product& q, dim3 grid) {
    hipLaunchKernelGGL((fp8_gemm_rows_kernel<MT, NT, W, P>), grid, dim3(64 * W), 0, stream, q);
  });
}

hipError_t launch_fp8_gemm(const Fp8Product& p, hipStream_t stream) {
  if (p.M <= 16) return launch_rows<1, 1, 8, 2>(p, stream);
  return launch_rows<4, 4, 4, 1>(p, stream);
}

}  // namespace nvfp4
