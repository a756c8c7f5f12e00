// Residual addition, RMS norm and 8-bit output with scales (definition:
// include/int4.h, int4_rmsnorm_quant8): h = x + r, y = h w / sqrt(mean h^2 +
// eps), s = max|y| / Q, code = round(y / s).
//
// One pass over memory: a team of T threads holds a row of h in registers
// (vectors of 8 columns, V a thread, thread t has vectors t, t + T, ...), adds
// up h^2 and takes the maximum of |h w|, neither of which needs the norm, and
// after one exchange multiplies h w by inv / s.  Groups of 32, 64 and 128
// columns are 4, 8 and 16 neighbouring lanes.
//
// A code is the nearest to the exact y / s, so sums, products and quotients
// are fp64 wherever fp32 would round: h^2 always, the rest where h or w is
// fp32.  With bf16 h and w the products h w are exact in fp32 unless they leave
// its range, and y / s in fp32 decides a code unless it is within its error of
// half way between two codes; only a wave that has such an element redoes its
// vectors in fp64, and where a maximum |h w| is next to either end of fp32's
// range (or 0, as it is where all products underflow) it is taken again in fp64.
//
// Bound by memory at long rows (4096 x 4096, bf16 with a bf16 residual, E4M3 in
// groups of 128: 118 MB in 23.7 us, 5.0 TB/s; a large copy runs at 5.1), with
// vector issue behind it (34 instructions an element there are 15 us, 22 with
// one INT8 scale a row); 110593 x 128 to INT8: 43 MB in 10.0 us, 11.6 from memory.
#include <type_traits>

#include "device_common.hpp"
#include "encode8.hpp"
#include "int4_kernels.hpp"
#include "lanes.hpp"

namespace nvfp4 {

enum class Res { kNone, kBf16, kF32 };

// 1 / sqrt(x) for positive normal x, as rcp64.
__device__ __forceinline__ double rsqrt64(double x) {
  double y = __builtin_amdgcn_rsq(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __builtin_fma(y, __builtin_fma(-0.5 * x * y, y, 0.5), y);
  return y;
}

template <bool WBF>
__device__ __forceinline__ void load_weight(const NormArgs& a, int i, Vec8<WBF>& w) {
  if (a.weight) {
    w.load(a.weight, i);
  } else {  // ones
    const uint32_t one = WBF ? 0x3F803F80u : 0x3F800000u;
    w.a[0] = u32x4{one, one, one, one};
    w.a[WBF ? 0 : 1] = w.a[0];
  }
}

template <int T, int V, bool XBF, Res RES, bool WBF>
__global__ __launch_bounds__(T < 256 ? 256 : T, T >= 512 ? (V <= 2 ? 8 : 4) : 1) void rmsnorm_quant_kernel(
    NormArgs a, double inv_cols, double inv_top) {
  constexpr int B = T < 256 ? 256 : T, TEAMS = B / T, NW = T / 64;
  const int t = threadIdx.x % T;
  const int64_t r = (int64_t)blockIdx.x * TEAMS + threadIdx.x / T;
  const int n8 = a.cols / 8;
  const bool live_row = r < a.rows;
  // Where a thread has many vectors the weight, and then h too, is read again
  // for the codes (a cache hit; the registers are worth more: two workgroups
  // of 1024 threads a CU instead of one take 2000 x 14336 from 50 to 43 us, 400
  // x 28672 in bf16 from 21.9 to 20.5; in fp32, twice the bytes, keeping h is
  // faster there, 38.7 to 42.2).
  constexpr bool HBF = RES == Res::kNone ? XBF : RES == Res::kBf16;
  constexpr bool kKeep = V <= (T == 1024 ? 1 : 2), kKeepH = V <= (HBF ? 2 : 4);
  constexpr bool kFast = HBF && WBF;
  using Max = typename std::conditional<kFast, float, double>::type;
  Vec8<HBF> h[kKeepH ? V : 1];
  Vec8<WBF> w[kKeep ? V : 1];
  double ss = 0.0;
  // Maximum |h w| of each vector; where h is not kept one for all of them, and
  // the groups' are taken again.
  constexpr int kUnroll = kKeepH ? V : 1;
  Max m[kUnroll] = {};
  const auto top_of = [](const Vec8<HBF>& hv, const Vec8<WBF>& wv, Max top) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (kFast) top = fmaxf(top, fabsf(hv.at(j) * wv.at(j)));
      else top = fmax(top, fabs((double)hv.at(j) * (double)wv.at(j)));
    }
    return top;
  };
  // Where fp32 products serve: the maximum far from overflow, and so far above
  // fp32's smallest that products which lose bits there are neither the maximum
  // nor more than code 0.
  const auto in_range = [](float top) { return top >= 0x1p-100f && top <= 0x1p126f; };
  // Maximum |h w| of vector v in fp64, of h and the weight as they lie in
  // memory: kept in registers for this rare path, they would cost a wave a
  // SIMD.
  const auto wide_top_of = [&](int v) {
    const int i = fresh(t + T * v);
    double top = 0.0;
    if (live_row && i < n8) {
      Vec8<HBF> hv;
      Vec8<WBF> wv;
      if constexpr (RES == Res::kNone) hv.load(a.x, r * a.x_stride + 8 * i);
      else hv.load(a.residual_out, r * a.cols + 8 * i);
      load_weight<WBF>(a, 8 * i, wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmax(top, fabs((double)hv.at(j) * (double)wv.at(j)));
    }
    return top;
  };
  __shared__ double red_ss[16];
  __shared__ Max red_max[16];
#pragma unroll kUnroll
  for (int v = 0; v < V; ++v) {
    const int i = t + T * v;
    Vec8<WBF>& wv = w[kKeep ? v : 0];
    Vec8<HBF>& hv = h[kKeepH ? v : 0];
    hv.zero();
    wv.zero();
    if (live_row && i < n8) {
      if constexpr (RES == Res::kNone) {
        hv.load(a.x, r * a.x_stride + 8 * i);
      } else {
        Vec8<XBF> x;
        x.load(a.x, r * a.x_stride + 8 * i);
        hv.load(a.residual, r * a.res_stride + 8 * i);
        float sum[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = x.at(j) + hv.at(j);
        hv.set(sum);
        hv.store(a.residual_out, r * a.cols + 8 * i);
      }
      load_weight<WBF>(a, 8 * i, wv);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)hv.at(j), (double)hv.at(j), ss);
    m[v % kUnroll] = top_of(hv, wv, m[v % kUnroll]);
    if (V > 2) __builtin_amdgcn_sched_barrier(0);  // one vector's operands at a time
  }
  const auto add = [](double p, double q) { return p + q; };
  const auto most = [](auto p, auto q) { return p > q ? p : q; };
  Max all = 0;  // the row's maximum
  if (a.group == 0) {
#pragma unroll
    for (int v = 0; v < kUnroll; ++v) all = most(all, m[v]);
  }
  constexpr int W = T < 64 ? T : 64;
  ss = lanes_all<W>(ss, add);
  if (a.group == 0) all = lanes_all<W>(all, most);
  if constexpr (T > 64) {
    // every lane reads the partial results, which each run of 4, 8 or 16 lanes
    // (as many as waves) then combines in the same way
    const int wave = threadIdx.x / 64;
    if (threadIdx.x % 64 == 0) {
      red_ss[wave] = ss;
      red_max[wave] = all;
    }
    __syncthreads();
    ss = red_ss[threadIdx.x % NW];
    ss = lanes_all<NW>(ss, add);
    if (a.group == 0) {
      all = red_max[threadIdx.x % NW];
      all = lanes_all<NW>(all, most);
    }
  }
  const double ms = __builtin_fma(ss, inv_cols, a.eps);
  const double inv = ms > 0.0 ? rsqrt64(ms) : 0.0;
  const int L = a.group / 8, Ls = 31 - __builtin_clz(L | 1), G = a.group ? (a.cols + a.group - 1) / a.group : 1;
  // scale, and the factor that turns h w into y / s
  const auto scale_of = [&](double top, float& s) {
    s = (float)(top * inv * inv_top);
    if (s == 0.0f) s = 1.0f;
    return inv * rcp64((double)s);
  };
  float s_row = 1.0f;
  double k = 0.0;
  if (a.group == 0) {
    double top = (double)all;
    if constexpr (kFast) {
      // the same for all threads of the row (a maximum of fmaxf's, so never NaN)
      if (!in_range(all)) {
        top = 0.0;
#pragma unroll 1
        for (int v = 0; v < V; ++v) top = most(top, wide_top_of(v));
        top = lanes_all<W>(top, most);
        if constexpr (T > 64) {  // a row is a workgroup
          __syncthreads();       // red_ss has been read
          if (threadIdx.x % 64 == 0) red_ss[threadIdx.x / 64] = top;
          __syncthreads();
          top = lanes_all<NW>(red_ss[threadIdx.x % NW], most);
        }
      }
    }
    k = scale_of(top, s_row);
    if (t == 0 && live_row) a.scales[r] = s_row;
  }
#pragma unroll kUnroll
  for (int v = 0; v < V; ++v) {
    const int i = t + T * v;
    const bool live = live_row && i < n8;
    Vec8<WBF>& wv = w[kKeep ? v : 0];
    Vec8<HBF>& hv = h[kKeepH ? v : 0];
    if constexpr (!kKeepH) {
      hv.zero();
      wv.zero();
    }
    if (live) {
      if (!kKeep) load_weight<WBF>(a, 8 * i, wv);
      if constexpr (!kKeepH) {
        if constexpr (RES == Res::kNone) hv.load(a.x, r * a.x_stride + 8 * i);
        else hv.load(a.residual_out, r * a.cols + 8 * i);
      }
    }
    Max top = all;
    float s = s_row;
    if (a.group) {
      top = lanes_all(kKeepH ? m[v % kUnroll] : top_of(hv, wv, 0), L, most);
      double wide = (double)top;
      if constexpr (kFast) {
        // the same for the L lanes of a group
        if (!in_range(top)) wide = lanes_all(wide_top_of(v), L, most);
      }
      k = scale_of(wide, s);
      if (live && (i & (L - 1)) == 0) a.scales[r * G + (i >> Ls)] = s;
    }
    if (live) {
      u32x2 q;
      bool exact = true;
      if constexpr (kFast) {
        // s normal, so |u| stays below Q and half a step
        exact = !(in_range(top) && s >= 0x1p-120f);
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = hv.at(j) * wv.at(j);
        if (a.e4m3) {
          double d[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] = (double)p[j];
          q = encode_e4m3(d, k);
        } else {
          q = encode_i8_fast(p, (float)k, exact);
        }
      }
      if (exact) {
        double p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          p[j] = kFast ? (double)fresh(hv.at(j)) * (double)fresh(wv.at(j)) : (double)hv.at(j) * (double)wv.at(j);
        q = a.e4m3 ? encode_e4m3(p, k) : encode_i8(p, k);
      }
      *reinterpret_cast<u32x2*>(reinterpret_cast<uint8_t*>(a.codes) + r * a.cols + 8 * i) = q;
    }
    if (V > 2) __builtin_amdgcn_sched_barrier(0);
  }
}

// Threads a row and vectors a thread, by the row's length, from a sweep over
// both: the fewest vectors a thread without teams that are mostly idle.  (us:
// 4096 x 4096, 512 x 1 25.2, 256 x 2 25.7, 1024 x 1 27.5, 256 x 4 29.6; 300 x 4096,
// 512 x 1 4.3, 256 x 2 4.6, 1024 x 1 4.9; 2048 x 8192, 1024 x 1 26.3, 512 x 2 28.0;
// 2000 x 14336, 1024 x 2 43.7, 512 x 4 46.6; 16384 x 1024, 64 x 2 24.8, 256 x 1
// 29.3.)
template <bool XBF, Res RES, bool WBF>
hipError_t launch_norm(const NormArgs& all, hipStream_t stream) {
  const int n8 = all.cols / 8, G = all.group ? (all.cols + all.group - 1) / all.group : 1;
  const double ic = 1.0 / all.cols, it = all.e4m3 ? 1.0 / 448.0 : 1.0 / 127.0;
  constexpr int HB = RES == Res::kNone ? 0 : RES == Res::kBf16 ? 2 : 4;  // bytes of a residual
  // at most 2^20 workgroups a launch (a launch counts its threads in 32 bits)
  const int64_t step = ((int64_t)1 << 20) * (n8 <= 16 ? 16 : n8 <= 128 ? 4 : 1);
  for (int64_t r0 = 0; r0 < all.rows; r0 += step) {
    NormArgs a = all;
    a.rows = all.rows - r0 < step ? all.rows - r0 : step;
    a.x = reinterpret_cast<const char*>(all.x) + r0 * all.x_stride * (XBF ? 2 : 4);
    if (RES != Res::kNone) {
      a.residual = reinterpret_cast<const char*>(all.residual) + r0 * all.res_stride * HB;
      a.residual_out = reinterpret_cast<char*>(all.residual_out) + r0 * all.cols * HB;
    }
    a.codes = reinterpret_cast<char*>(all.codes) + r0 * all.cols;
    a.scales = all.scales + r0 * G;
#define NORM_CASE(T, V)                                                                                  \
  hipLaunchKernelGGL((rmsnorm_quant_kernel<T, V, XBF, RES, WBF>),                                        \
                     dim3((unsigned)((a.rows + (T < 256 ? 256 / T : 1) - 1) / (T < 256 ? 256 / T : 1))), \
                     dim3(T < 256 ? 256 : T), 0, stream, a, ic, it)
    if (n8 <= 16) NORM_CASE(16, 1);
    else if (n8 <= 64) NORM_CASE(64, 1);
    else if (n8 <= 128) NORM_CASE(64, 2);
    else if (n8 <= 256) NORM_CASE(256, 1);
    else if (n8 <= 512) NORM_CASE(512, 1);
    else if (n8 <= 1024) NORM_CASE(1024, 1);
    else if (n8 <= 2048) NORM_CASE(1024, 2);
    else if (n8 <= 4096) NORM_CASE(1024, 4);
    else NORM_CASE(1024, 8);
#undef NORM_CASE
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool XBF, Res RES>
hipError_t launch_norm_w(const NormArgs& a, hipStream_t stream) {
  // no weight counts as bf16 (ones)
  return !a.weight || a.w_bf16 ? launch_norm<XBF, RES, true>(a, stream) : launch_norm<XBF, RES, false>(a, stream);
}

hipError_t launch_rmsnorm_quant8(const NormArgs& a, hipStream_t stream) {
  if (!a.residual)
    return a.x_bf16 ? launch_norm_w<true, Res::kNone>(a, stream) : launch_norm_w<false, Res::kNone>(a, stream);
  if (a.res_bf16) return launch_norm_w<true, Res::kBf16>(a, stream);
  return a.x_bf16 ? launch_norm_w<true, Res::kF32>(a, stream) : launch_norm_w<false, Res::kF32>(a, stream);
}

}  // namespace nvfp4
