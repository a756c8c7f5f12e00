// Paged 8-bit caches of keys and values: quantized as they are written, and
// read back (definitions: include/kvcache.h).
//
// A workgroup has some tokens of one of the two tensors.  First a thread a
// token finds its place (a search in cu and one page number), then all threads
// move the tokens' heads, several vectors in flight each.  Memory bounds both
// where there are many tokens (65536 tokens of 8 heads of 128, bf16: written
// in 92 to 95 us, 4.3 to 4.4 TB/s, read in 87, 4.7; fp32 written in 138, 4.9, read in
// 194, 3.5), and below about a thousand the launch and the three reads that
// follow each other (cu, page number, codes): 4.5 us.
// (Every thread finding its own place and moving one vector: 137 us.)
#include "device_common.hpp"
#include "encode8.hpp"
#include "fp8_kernels.hpp"
#include "kv_search.hpp"
#include "lanes.hpp"

namespace nvfp4 {

constexpr int kMaxTokens = 256;  // of a workgroup

// Where a token is: page and row in the page; page -1 where it has no place,
// -2 where it belongs to no sequence.
struct Place {
  int page, row;
};
struct Places {
  Place at[kMaxTokens];
  int cu[kCuHeld + 1];  // (256 or fewer sequences are searched in LDS alone)
};

__device__ __forceinline__ Place locate(const kv8_places& p, const int* cu, int64_t t) {
  int first;
  const int64_t b = sequence_of(cu, [&](int64_t i) { return p.cu[i]; }, p.seqs, t, first);
  if (b < 0) return {-2, 0};
  const int64_t at = t - first + (p.starts ? p.starts[b] : 0);
  if (at < 0 || at >= p.table_width * p.page_size) return {-1, 0};
  const uint32_t slot = (uint32_t)at / (uint32_t)p.page_size;  // at < 2^32
  const int page = p.page_table[b * p.table_width + slot];
  return {page >= 0 && page < p.pages ? page : -1, (int)((uint32_t)at - slot * (uint32_t)p.page_size)};
}

// The places of this workgroup's tokens t0, t0 + 1, ..., and how many it has.
__device__ __forceinline__ int locate_all(const kv8_places& p, int64_t t0, int per_block, Places& places) {
  const int n = (int)min((int64_t)per_block, p.tokens - t0), k = threadIdx.x;
  places.cu[k] = p.cu[cu_entry(k, p.seqs)];
  if (k == 0) places.cu[kCuHeld] = p.cu[p.seqs];
  __syncthreads();
  if (k < n) places.at[k] = locate(p, places.cu, t0 + k);
  __syncthreads();
  return n;
}

// a / b for a < 2^31, with per = 2^32 / b rounded down (b > 1).
__device__ __forceinline__ uint32_t divide(uint32_t a, uint32_t b, uint32_t per) {
  if (b == 1) return a;
  const uint32_t q = __umulhi(a, per);  // exact or one short
  return q + (a - q * b >= b ? 1 : 0);
}

// A row is one token and head; T lanes have it, 16 elements each (8191 tokens of
// 8 heads of 128, INT8: 13.7 us, with 8 elements 16.8), and U rows at a time.
// The maximum is fp32's, exact; the quotients are decided as encode8.hpp says.
template <bool BF, int T, int U>
__global__ __launch_bounds__(256) void kv8_write_kernel(kv8_tensor keys, kv8_tensor values, kv8_places p, bool e4m3,
                                                        int64_t first, int per_block, uint32_t per_head) {
  __shared__ Places places;
  const kv8_tensor& c = blockIdx.y ? values : keys;
  const int64_t t0 = first + (int64_t)blockIdx.x * per_block;
  const int n = locate_all(p, t0, per_block, places) * (int)p.heads;
  const int lane = threadIdx.x % T, e = 16 * lane;
  const double q = e4m3 ? 448.0 : 127.0, inv_q = e4m3 ? 1.0 / 448.0 : 1.0 / 127.0;
  for (int i0 = threadIdx.x / T; i0 < n; i0 += U * (256 / T)) {
    Vec8<BF> v[U][2];
    uint8_t* codes[U];
    float* scale[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * (256 / T);
      codes[u] = nullptr;
      v[u][0].zero();
      v[u][1].zero();
      if (i < n) {
        const int t = (int)divide((uint32_t)i, (uint32_t)p.heads, per_head), h = i - t * (int)p.heads;
        const Place at = places.at[t];
        if (at.page >= 0) {  // the same for the T lanes
          const int64_t row = (int64_t)at.row * p.heads + h;
          codes[u] = reinterpret_cast<uint8_t*>(c.codes) + at.page * c.code_stride + row * c.dim + e;
          scale[u] = c.scales + at.page * c.scale_stride + row;
          if (e < c.dim) {
            const int64_t from = (t0 + t) * c.token_stride + h * c.head_stride + e;
            v[u][0].load(c.rows, from);
            v[u][1].load(c.rows, from + 8);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!codes[u]) continue;
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(v[u][k / 8].at(k % 8)));
      const auto most = [](float a, float b) { return fmaxf(a, b); };
      if (T > 1) top = most(top, dpp<kDppXor1>(top));
      if (T > 2) top = most(top, dpp<kDppXor2>(top));
      if (T > 4) top = most(top, dpp<kDppHalfMirror>(top));
      if (T > 8) top = most(top, dpp<kDppMirror>(top));
      if (T > 16) top = most(top, __shfl_xor(top, 16));
      if (T > 32) top = most(top, __shfl_xor(top, 32));
      float s = (float)quotient((double)top, q, inv_q);
      s = s == 0.0f ? 1.0f : s;
      if (lane == 0) *scale[u] = s;
      if (e < c.dim) {
        const u32x2 a = encode(v[u][0], s, e4m3), b = encode(v[u][1], s, e4m3);
        *reinterpret_cast<u32x4*>(codes[u]) = u32x4{a.x, a.y, b.x, b.y};
      }
    }
  }
}

// A thread has 16 elements of a head, U times.  scale * code is rounded to fp32
// once and from there to bf16, as the definition has it.
template <bool BF, int U>
__global__ __launch_bounds__(256) void kv8_read_kernel(kv8_tensor keys, kv8_tensor values, kv8_places p, bool e4m3,
                                                       int64_t first, int per_block, uint32_t per_k, uint32_t per_v,
                                                       uint32_t per_head) {
  __shared__ Places places;
  const kv8_tensor& c = blockIdx.y ? values : keys;
  const uint32_t units = (uint32_t)c.dim / 16, per_unit = blockIdx.y ? per_v : per_k;
  const int64_t t0 = first + (int64_t)blockIdx.x * per_block;
  const uint32_t n = (uint32_t)locate_all(p, t0, per_block, places) * (uint32_t)p.heads * units;
  for (uint32_t i0 = threadIdx.x; i0 < n; i0 += 256 * U) {
    u32x4 q[U];
    float s[U];
    int64_t at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = i0 + 256 * u;
      q[u] = u32x4{0, 0, 0, 0};  // no place: zeros
      s[u] = 0.0f;
      at[u] = -1;
      if (i < n) {
        const uint32_t head = divide(i, units, per_unit), t = divide(head, (uint32_t)p.heads, per_head);
        const uint32_t h = head - t * (uint32_t)p.heads, e = 16 * (i - head * units);
        const Place place = places.at[t];
        if (place.page != -2) at[u] = (t0 + t) * c.token_stride + h * c.head_stride + e;
        if (place.page >= 0) {
          const int64_t row = (int64_t)place.row * p.heads + h;
          s[u] = c.scales[place.page * c.scale_stride + row];
          q[u] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(c.codes) + place.page * c.code_stride +
                                                 row * c.dim + e);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (at[u] < 0) continue;
      float v[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (e4m3) {
          const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(q[u][j], false);
          const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(q[u][j], true);
          v[4 * j] = a.x * s[u], v[4 * j + 1] = a.y * s[u], v[4 * j + 2] = b.x * s[u], v[4 * j + 3] = b.y * s[u];
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) v[4 * j + k] = (float)(int8_t)(q[u][j] >> (8 * k)) * s[u];
        }
      }
      Vec8<BF> o;
      o.set(v);
      o.store(c.rows, at[u]);
      o.set(v + 8);
      o.store(c.rows, at[u] + 8);
    }
  }
}

hipError_t launch_kv8(const kv8_tensor& keys, const kv8_tensor& values, const kv8_places& p, bool bf16, bool e4m3,
                      bool write, hipStream_t stream) {
  const int64_t dim = keys.dim > values.dim ? keys.dim : values.dim;
  const auto per = [](int64_t d) { return d > 1 ? (uint32_t)(((uint64_t)1 << 32) / (uint64_t)d) : 0u; };
  const uint32_t per_head = per(p.heads);
  // Vectors a thread moves at a time: 4 where there are enough for 4 workgroups
  // a CU, otherwise 1; a workgroup has as many tokens as give its threads those
  // (at most 2^22 workgroups a launch, which counts its threads in 32 bits).
  const auto launch = [&](int64_t vectors_of_token, auto kernel) {
    const int64_t all = p.tokens * vectors_of_token;
    const int u = all >= 4 * 256 * 1024 ? 4 : 1;
    const int64_t fit = 256 * u / vectors_of_token;
    const int n = (int)(fit < 1 ? 1 : fit > kMaxTokens ? kMaxTokens : fit);
    const int64_t step = (int64_t)n << 22;
    for (int64_t first = 0; first < p.tokens; first += step) {
      const int64_t blocks = ((p.tokens - first < step ? p.tokens - first : step) + n - 1) / n;
      kernel(dim3((unsigned)blocks, 2), u, first, n);
      if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
  };
  if (!write) {
    return launch(p.heads * (dim / 16), [&](dim3 g, int u, int64_t first, int n) {
#define READ_CASE(BF, U)                                                                                   \
  hipLaunchKernelGGL((kv8_read_kernel<BF, U>), g, dim3(256), 0, stream, keys, values, p, e4m3, first, n,    \
                     per(keys.dim / 16), per(values.dim / 16), per_head)
      if (bf16 && u == 4) READ_CASE(true, 4);
      else if (bf16) READ_CASE(true, 1);
      else if (u == 4) READ_CASE(false, 4);
      else READ_CASE(false, 1);
#undef READ_CASE
    });
  }
#define WRITE_CASE(T)                                                                                           \
  launch(p.heads * T, [&](dim3 g, int u, int64_t first, int n) {                                                \
    const auto kernel = bf16 ? u == 4 ? kv8_write_kernel<true, T, 4> : kv8_write_kernel<true, T, 1>             \
                             : u == 4 ? kv8_write_kernel<false, T, 4> : kv8_write_kernel<false, T, 1>;          \
    hipLaunchKernelGGL(kernel, g, dim3(256), 0, stream, keys, values, p, e4m3, first, n, per_head);             \
  })
  if (dim <= 64) return WRITE_CASE(4);
  if (dim <= 128) return WRITE_CASE(8);
  if (dim <= 256) return WRITE_CASE(16);
  if (dim <= 512) return WRITE_CASE(32);
  return WRITE_CASE(64);
#undef WRITE_CASE
}

}  // namespace nvfp4
