// Paged 8-bit caches of keys and values: quantized as they are written, and
// read back (definitions: include/kvcache.h).
#include "device_common.hpp"
#include "encode8.hpp"
#include "fp8_kernels.hpp"
#include "lanes.hpp"

namespace nvfp4 {

enum class Place { kHeld, kNowhere, kNoSequence };

// Where row t belongs: page and row in the page.
__device__ __forceinline__ Place locate(const kv8_places& p, int64_t t, int64_t& page, int64_t& row) {
  int lo = 0, hi = (int)p.seqs;
  if (t < p.cu[0] || t >= p.cu[hi]) return Place::kNoSequence;
  while (hi - lo > 1) {  // cu[lo] <= t < cu[hi]
    const int mid = lo + (hi - lo) / 2;
    if (p.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int64_t at = t - p.cu[lo] + (p.starts ? p.starts[lo] : 0);
  if (at < 0) return Place::kNowhere;
  const int64_t slot = at / p.page_size;
  if (slot >= p.table_width) return Place::kNowhere;
  page = p.page_table[lo * p.table_width + slot];
  row = at - slot * p.page_size;
  return page >= 0 && page < p.pages ? Place::kHeld : Place::kNowhere;
}

// A row is one token and head; T lanes have it, V vectors of 8 elements each.
template <bool BF, int T, int V>
__global__ __launch_bounds__(256) void kv8_write_kernel(kv8_tensor keys, kv8_tensor values, kv8_places p, bool e4m3) {
  const kv8_tensor& c = blockIdx.y ? values : keys;
  const int lane = threadIdx.x % T;
  const int64_t all = p.tokens * p.heads, step = (int64_t)gridDim.x * (256 / T);
  for (int64_t i = (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T; i < all; i += step) {
    const int64_t t = i / p.heads, h = i - t * p.heads;
    int64_t page, row;
    if (locate(p, t, page, row) != Place::kHeld) continue;  // the same for the T lanes
    Vec8<BF> v[V];
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[j].zero();
      const int e = 8 * (lane + T * j);
      if (e < c.dim) v[j].load(c.rows, t * c.token_stride + h * c.head_stride + e);
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[j].at(k)));
    }
    const auto most = [](float a, float b) { return fmaxf(a, b); };
    top = lanes_all<(T > 16 ? 16 : T)>(top, most);
    if (T >= 32) top = most(top, __shfl_xor(top, 16));
    if (T >= 64) top = most(top, __shfl_xor(top, 32));
    const float s = scale_for((double)top, e4m3 ? 448.0 : 127.0);
    const int64_t at = row * p.heads + h;
    if (lane == 0) c.scales[page * c.scale_stride + at] = s;
    uint8_t* codes = reinterpret_cast<uint8_t*>(c.codes) + page * c.code_stride + at * c.dim;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = 8 * (lane + T * j);
      double d[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = (double)v[j].at(k);
      if (e < c.dim) *reinterpret_cast<u32x2*>(codes + e) = encode_quotients(d, s, e4m3);
    }
  }
}

// A thread has 16 elements of a row.
template <bool BF>
__global__ __launch_bounds__(256) void kv8_read_kernel(kv8_tensor keys, kv8_tensor values, kv8_places p, bool e4m3) {
  const kv8_tensor& c = blockIdx.y ? values : keys;
  const int64_t per = c.dim / 16, all = p.tokens * p.heads * per, step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += step) {
    const int64_t u = i / per, t = u / p.heads, h = u - t * p.heads, e = 16 * (i - u * per);
    int64_t page, row;
    const Place place = locate(p, t, page, row);
    if (place == Place::kNoSequence) continue;
    float v[16] = {};
    if (place == Place::kHeld) {
      const int64_t at = row * p.heads + h;
      const float s = c.scales[page * c.scale_stride + at];
      const u32x4 q =
          *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(c.codes) + page * c.code_stride + at * c.dim + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (e4m3) {
          const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(q[j], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(q[j], true);
          v[4 * j] = a.x * s, v[4 * j + 1] = a.y * s, v[4 * j + 2] = b.x * s, v[4 * j + 3] = b.y * s;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) v[4 * j + k] = (float)(int8_t)(q[j] >> (8 * k)) * s;
        }
      }
    }
    const int64_t at = t * c.token_stride + h * c.head_stride + e;
    Vec8<BF> o;
    o.set(v);
    o.store(c.rows, at);
    o.set(v + 8);
    o.store(c.rows, at + 8);
  }
}

hipError_t launch_kv8(const kv8_tensor& keys, const kv8_tensor& values, const kv8_places& p, bool bf16, bool e4m3,
                      bool write, hipStream_t stream) {
  const int64_t dim = keys.dim > values.dim ? keys.dim : values.dim;
  const auto grid = [](int64_t blocks) { return dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20), 2); };
  if (!write) {
    const dim3 g = grid((p.tokens * p.heads * (dim / 16) + 255) / 256);
    if (bf16) hipLaunchKernelGGL(kv8_read_kernel<true>, g, dim3(256), 0, stream, keys, values, p, e4m3);
    else hipLaunchKernelGGL(kv8_read_kernel<false>, g, dim3(256), 0, stream, keys, values, p, e4m3);
    return hipGetLastError();
  }
#define WRITE_CASE(T, V)                                                                                             \
  do {                                                                                                               \
    const dim3 g = grid((p.tokens * p.heads + 256 / T - 1) / (256 / T));                                             \
    if (bf16)                                                                                                        \
      hipLaunchKernelGGL((kv8_write_kernel<true, T, V>), g, dim3(256), 0, stream, keys, values, p, e4m3);            \
    else                                                                                                             \
      hipLaunchKernelGGL((kv8_write_kernel<false, T, V>), g, dim3(256), 0, stream, keys, values, p, e4m3);           \
  } while (0)
  if (dim <= 64) WRITE_CASE(8, 1);
  else if (dim <= 128) WRITE_CASE(16, 1);
  else if (dim <= 256) WRITE_CASE(32, 1);
  else if (dim <= 512) WRITE_CASE(64, 1);
  else WRITE_CASE(64, 2);
#undef WRITE_CASE
  return hipGetLastError();
}

}  // namespace nvfp4
