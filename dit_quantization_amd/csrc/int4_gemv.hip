// Decode products y = x W^T for group-scaled 4-bit integer weights and bf16,
// INT8 or E4M3 activations, M <= 16 rows (format: include/int4.h):
//   y[m, n] = sum_g s[n, g] sx[m, g] (sum_{k in g} x c - z[n, g] sum_{k in g} x)
// The codes c = 0..15 go into the products as they are: a mask and a shift
// turn 8 nibbles into 8 bytes, and such a byte is at once the INT8 value c
// and the E4M3 value c / 512 (subnormals and the first binade are evenly
// spaced).  INT8 activations meet them in integer products (exact inside a
// group); for bf16 and E4M3 ones the FP8 converter makes exact bf16 pairs
// c / 512, and the 512 goes into the scale.  The zero point is taken
// off with the sum of x, which all rows of the weight share.
#include "device_common.hpp"
#include "int4_kernels.hpp"

namespace nvfp4 {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// What a product of bytes has to be multiplied by.
template <Act A>
constexpr float kUnit = A == Act::kI8 ? 1.0f : 512.0f;

constexpr uint32_t kNibbles = 0x0F0F0F0Fu;

// ---- one row (M = 1): dot products on the vector units.
// A workgroup of 4 waves: S waves split K, the 4 / S wave groups take RW rows
// each.  Lane l of a wave has the 16-byte chunks (32 codes, inside one group)
// l, l + 64, ... of its K part, so one load instruction reads 1 KB of a row,
// and keeps the x of its chunks and their sums in registers for all its rows.
// Loads past the K part, or of rows past N, return zeros.
template <Act A>
struct Chunk {             // x of one chunk
  uint32_t x[A == Act::kI8 ? 8 : 16];
  float sum;               // in units of the code products
  float scale;
};

__device__ __forceinline__ float dot2_bf16(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
}
__device__ __forceinline__ uint32_t pk_bf16_e4m3(uint32_t w, bool high) {
  return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                                           : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}

template <Act A>
__device__ __forceinline__ void load_chunk(Chunk<A>& c, __amdgpu_buffer_rsrc_t xbuf, int chunk, bool ok) {
  constexpr int BYTES = A == Act::kBf16 ? 64 : 32;
  uint32_t raw[BYTES / 4];
#pragma unroll
  for (int q = 0; q < BYTES / 16; ++q) {
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(xbuf, ok ? BYTES * chunk + 16 * q : kBufOOB, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) raw[4 * q + j] = v[j];
  }
  if constexpr (A == Act::kI8) {
    int s = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c.x[j] = raw[j];
      s = __builtin_amdgcn_sdot4((int)raw[j], 0x01010101, s, false);
    }
    c.sum = (float)s;
  } else {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      c.x[j] = A == Act::kBf16 ? raw[j] : pk_bf16_e4m3(raw[j / 2 % (BYTES / 4)], j & 1);
      s = dot2_bf16(c.x[j], 0x3B003B00u, s);  // 2^-9 each
    }
    c.sum = s;
  }
}

// sum over a chunk of x (code - z), in kUnit
template <Act A>
__device__ __forceinline__ float dot_chunk(const Chunk<A>& c, u32x4 w, float z) {
  if constexpr (A == Act::kI8) {
    int p = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      p = __builtin_amdgcn_sdot4((int)c.x[2 * d], (int)(w[d] & kNibbles), p, false);
      p = __builtin_amdgcn_sdot4((int)c.x[2 * d + 1], (int)((w[d] >> 4) & kNibbles), p, false);
    }
    return __builtin_fmaf(-z, c.sum, (float)p);  // whole numbers below 2^24: exact
  } else {
    float p[2] = {0.0f, 0.0f};
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t lo = w[d] & kNibbles, hi = (w[d] >> 4) & kNibbles;
      p[d & 1] = dot2_bf16(c.x[4 * d], pk_bf16_e4m3(lo, false), p[d & 1]);
      p[d & 1] = dot2_bf16(c.x[4 * d + 1], pk_bf16_e4m3(lo, true), p[d & 1]);
      p[d & 1] = dot2_bf16(c.x[4 * d + 2], pk_bf16_e4m3(hi, false), p[d & 1]);
      p[d & 1] = dot2_bf16(c.x[4 * d + 3], pk_bf16_e4m3(hi, true), p[d & 1]);
    }
    return __builtin_fmaf(-z, c.sum, p[0] + p[1]);
  }
}

// Sum of v[r] over the 64 lanes for every r < R; lane l ends with the total
// of row l % R (R = 1, 2 or 4).
template <int R>
__device__ __forceinline__ float lane_sums(float (&v)[R], int lane) {
#pragma unroll
  for (int half = R / 2; half > 0; half /= 2) {
    const bool upper = (lane & half) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i)
      v[i] = (upper ? v[i + half] : v[i]) + __shfl_xor(upper ? v[i] : v[i + half], half);
  }
#pragma unroll
  for (int o = R; o < 64; o *= 2) v[0] += __shfl_xor(v[0], o);
  return v[0];
}

template <Act A, int CH, int RW, int S>
__global__ __launch_bounds__(256) void int4_gemv_m1_kernel(Int4Act x, Int4Weight w, int shift, int N, int K, int G,
                                                           void* __restrict__ y, int bf16_out) {
  constexpr int GROUPS = 4 / S;
  __shared__ float red[4][RW];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % S, grp = wave / S;
  const int nch = K / 32, per = (nch + S - 1) / S;
  const int cbeg = part * per, cend = min(cbeg + per, nch);
  const int row0 = (blockIdx.x * GROUPS + grp) * RW;
  const int nrows = __builtin_amdgcn_readfirstlane(max(0, min(RW, N - row0)));
  const int64_t rb = min(row0, N - 1);
  const __amdgpu_buffer_rsrc_t cbuf = make_buf(w.codes + rb * (K / 2), (uint32_t)(nrows * (K / 2)));
  const __amdgpu_buffer_rsrc_t sbuf = make_buf(w.scales + rb * G, (uint32_t)(nrows * G * 2));
  const __amdgpu_buffer_rsrc_t zbuf = make_buf(w.zeros ? w.zeros + rb * G : nullptr, w.zeros ? (uint32_t)(nrows * G) : 0u);
  const __amdgpu_buffer_rsrc_t xbuf = make_buf(x.x, (uint32_t)(K * (A == Act::kBf16 ? 2 : 1)));
  u32x4 cw[RW][CH];
  uint32_t sw[RW][CH], zw[RW][CH];
  Chunk<A> xc[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int ch = cbeg + lane + 64 * c;
    load_chunk<A>(xc[c], xbuf, ch, ch < cend);
    xc[c].scale = A != Act::kBf16 && x.grouped && ch < cend ? x.scales[ch >> shift] : 1.0f;
  }
#pragma unroll
  for (int r = 0; r < RW; ++r) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = cbeg + lane + 64 * c;
      const bool ok = ch < cend;
      cw[r][c] = __builtin_amdgcn_raw_buffer_load_b128(cbuf, ok ? r * (K / 2) + 16 * ch : kBufOOB, 0, kBufNT);
      const int slot = r * G + (ch >> shift);
      sw[r][c] = __builtin_amdgcn_raw_buffer_load_b16(sbuf, ok ? 2 * slot : kBufOOB, 0, 0);
      zw[r][c] = w.zeros ? __builtin_amdgcn_raw_buffer_load_b8(zbuf, ok ? slot : kBufOOB, 0, 0) : 8u;
    }
    __builtin_amdgcn_sched_barrier(0);  // issue order = row order
  }
  float acc[RW];
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    acc[r] = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      acc[r] = __builtin_fmaf(dot_chunk<A>(xc[c], cw[r][c], (float)zw[r][c]),
                              bf16_bits_to_f32(sw[r][c]) * xc[c].scale, acc[r]);
    __builtin_amdgcn_sched_barrier(0);  // compute order = row order
  }
  const float tot = lane_sums<RW>(acc, lane);
  if (lane < RW) red[wave][lane] = tot;
  __syncthreads();
  if (threadIdx.x < GROUPS * RW) {
    const int g = threadIdx.x / RW, r = threadIdx.x % RW;
    float sum = red[g * S][r];
#pragma unroll
    for (int p = 1; p < S; ++p) sum += red[g * S + p][r];
    const int row = (blockIdx.x * GROUPS + g) * RW + r;
    sum *= kUnit<A> * (A != Act::kBf16 && !x.grouped ? x.scales[0] : 1.0f);
    if (row < N) {
      if (bf16_out)
        reinterpret_cast<uint16_t*>(y)[row] = (uint16_t)f32_to_bf16_bits(sum);
      else
        reinterpret_cast<float*>(y)[row] = sum;
    }
  }
}

// ---- several rows: 16 x 16 x 32 matrix instructions.
// A workgroup of NW waves owns 16 T weight rows; its waves split K into runs
// of super-chunks of 128 codes, 4 to a pass.  The codes of a pass reach LDS by
// DMA, every instruction reading 4 rows x 256 contiguous bytes, and lane
// (n, g) (n = lane % 16, g = lane / 16) reads back the 32 codes of chunk
// 4 s + g of row n from a row-swizzled slot.  A matrix instruction adds up
// over the lane groups g, so the codes it takes must be of one scale group:
// with groups of 128 those are the four lanes' chunks as they are; for 64 and
// 32 the dwords trade places between lane groups (v_permlane32_swap,
// v_permlane16_swap: a step each of a 4 x 4 transpose), after which
// instruction j covers chunks 2 (j / 2) + {0, 1}, or chunk j alone.  A
// product of one scale group starts at zero and is added into the fp32 sums
// with its scale, z taken off with the sums of x (one more matrix product
// with a constant operand, shared by the T row tiles).
//
// E4M3 activations are widened to bf16 as well: the FP8 matrix instruction
// keeps too few bits of its sums (9e-5 off, relative, after 160 products,
// where the bf16 one is off by less than 1e-6).
template <Act A>
struct Mfma {
  using Acc = f32x4;
  using X = u32x4;   // 8 bf16
  static constexpr int kBytes = A == Act::kBf16 ? 16 : 8;  // of 8 activations in memory
  static __device__ __forceinline__ Acc mul(X x, X w, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, w), c, 0, 0,
                                                   0);
  }
  static __device__ __forceinline__ X bytes(uint32_t a, uint32_t b) {
    return X{pk_bf16_e4m3(a, false), pk_bf16_e4m3(a, true), pk_bf16_e4m3(b, false), pk_bf16_e4m3(b, true)};
  }
  static __device__ __forceinline__ X unpack(uint32_t w) { return bytes(w & kNibbles, (w >> 4) & kNibbles); }
  static __device__ __forceinline__ X load(__amdgpu_buffer_rsrc_t buf, int off) {
    if constexpr (A == Act::kBf16) {
      return __builtin_amdgcn_raw_buffer_load_b128(buf, off, 0, 0);
    } else {
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(buf, off, 0, 0);
      return bytes(v.x, v.y);
    }
  }
  static __device__ __forceinline__ X ones() { return X{0x3B003B00u, 0x3B003B00u, 0x3B003B00u, 0x3B003B00u}; }
};
template <>
struct Mfma<Act::kI8> {
  using Acc = i32x4;
  using X = u32x2;
  static constexpr int kBytes = 8;
  static __device__ __forceinline__ Acc mul(X x, X w, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, x), __builtin_bit_cast(long, w), c, 0, 0, 0);
  }
  static __device__ __forceinline__ X unpack(uint32_t w) { return X{w & kNibbles, (w >> 4) & kNibbles}; }
  static __device__ __forceinline__ X load(__amdgpu_buffer_rsrc_t buf, int off) {
    return __builtin_amdgcn_raw_buffer_load_b64(buf, off, 0, 0);
  }
  static __device__ __forceinline__ X ones() { return X{0x01010101u, 0x01010101u}; }
};

// The dwords of lane (n, g)'s chunk become those its matrix instructions
// j = 0..3 take (see above).
template <int GS>
__device__ __forceinline__ u32x4 regroup(u32x4 d) {
  if constexpr (GS <= 64) {
    const auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    d = u32x4{a[0], b[0], a[1], b[1]};
  }
  if constexpr (GS == 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(d[0], d[1], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(d[2], d[3], false, false);
    d = u32x4{a[0], a[1], b[0], b[1]};
  }
  return d;
}

template <int G>
__device__ __forceinline__ void wait_newer(int k) {
  if (k == 0) __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
  else if (k == 1) __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(G));
  else if (k == 2) __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(2 * G));
  else __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(3 * G));
}

template <Act A, int GS, int T, int NW>
__global__ __launch_bounds__(NW * 64) void int4_gemv_mfma_kernel(Int4Act x, Int4Weight w, int M, int N, int K, int G,
                                                                 int wide, void* __restrict__ y, int bf16_out) {
  using Op = Mfma<A>;
  using Acc = typename Op::Acc;
  constexpr int SW = 4;           // super-chunks per pass
  constexpr int PER = 128 / GS;   // scale groups of a super-chunk
  constexpr int NG = SW * PER;    // and of a pass
  __shared__ u32x4 lds_c[NW][T][256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * (16 * T);
  const int rows = min(16 * T, N - n0);
  const int half = K / 2;
  const __amdgpu_buffer_rsrc_t cbuf = make_buf(w.codes + (int64_t)n0 * half, (uint32_t)(rows * half));
  const __amdgpu_buffer_rsrc_t sbuf = make_buf(w.scales + (int64_t)n0 * G, (uint32_t)(rows * G * 2));
  const __amdgpu_buffer_rsrc_t zbuf = make_buf(w.zeros ? w.zeros + (int64_t)n0 * G : nullptr,
                                               w.zeros ? (uint32_t)(rows * G) : 0u);
  const __amdgpu_buffer_rsrc_t xbuf = make_buf(x.x, (uint32_t)(M * K * (Op::kBytes / 8)));
  const bool grouped = A != Act::kBf16 && x.grouped;
  const __amdgpu_buffer_rsrc_t fbuf = make_buf(x.scales, grouped ? (uint32_t)(M * G * 4) : 0u);
  const int nch = K / 32, nsc = (nch + 3) / 4;
  const int per = ((nsc + NW - 1) / NW + SW - 1) / SW * SW;  // whole passes, so scales are read in aligned runs
  const int sbeg = wave * per, send = min(sbeg + per, nsc);

  f32x4 acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int s0 = sbeg; s0 < send; s0 += SW) {  // wave-uniform
    // x (L2 hits), then scales, then codes, so that what comes first is waited for first
    typename Op::X xa[SW][4];
#pragma unroll
    for (int u = 0; u < SW; ++u) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // the codes instruction j has from lane group g
        const int chunk = 4 * (s0 + u) + (GS == 128 ? g : GS == 64 ? 2 * (j >> 1) + (g & 1) : j);
        const int dword = GS == 128 ? j : GS == 64 ? 2 * (g >> 1) + (j & 1) : g;
        const bool ok = nl < M && chunk < nch && s0 + u < send;
        const int off = ok ? nl * (K * (Op::kBytes / 8)) + Op::kBytes * (4 * chunk + dword) : kBufOOB;
        xa[u][j] = Op::load(xbuf, off);
      }
    }
    const int g0 = s0 * PER;  // first scale group of the pass
    uint32_t sw[T][NG / 2], zw[T][NG / 4];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int base = (16 * t + nl) * G + g0;
      if (wide) {  // K % 512 == 0 and aligned pointers: the pass's groups lie inside the row
#pragma unroll
        for (int q = 0; q < NG / 4; ++q) {
          const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(sbuf, 2 * base + 8 * q, 0, 0);
          sw[t][2 * q] = v.x;
          sw[t][2 * q + 1] = v.y;
          zw[t][q] = w.zeros ? __builtin_amdgcn_raw_buffer_load_b32(zbuf, base + 4 * q, 0, 0) : 0x08080808u;
        }
      } else {
#pragma unroll
        for (int q = 0; q < NG / 2; ++q) sw[t][q] = 0;
#pragma unroll
        for (int q = 0; q < NG / 4; ++q) zw[t][q] = 0;
#pragma unroll
        for (int q = 0; q < NG; ++q) {
          const bool ok = g0 + q < G;
          sw[t][q / 2] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(sbuf, ok ? 2 * (base + q) : kBufOOB, 0, 0)
                          << (16 * (q & 1));
          zw[t][q / 4] |= (w.zeros ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(zbuf, ok ? base + q : kBufOOB, 0, 0) : 8u)
                          << (8 * (q & 3));
        }
      }
    }
    float fx[NG][4];
    if (grouped) {
#pragma unroll
      for (int q = 0; q < NG; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          fx[q][i] = __builtin_bit_cast(
              float, __builtin_amdgcn_raw_buffer_load_b32(
                         fbuf, 4 * g + i < M && g0 + q < G ? 4 * ((4 * g + i) * G + g0 + q) : kBufOOB, 0, 0));
    }
    // DMA instruction u of tile t fills LDS slots [64 u, 64 u + 64): lane l ->
    // row r = 4 u + l / 16, slot j = l % 16, holding chunk 4 s0 + (j ^ r).
    // Chunks past this wave's range, or past K, read as zero.
#pragma unroll
    for (int t = 0; t < T; ++t) {
      __builtin_amdgcn_sched_barrier(0);  // tile order
#pragma unroll
      for (int u = 0; u < SW; ++u) {
        const int r = 4 * u + (lane >> 4);
        const int c = 4 * s0 + ((lane & 15) ^ r);
        const bool ok = c < 4 * send && c < nch;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(cbuf, (__attribute__((address_space(3))) void*)&lds_c[wave][t][64 * u],
                                                 16, ok ? (16 * t + r) * half + 16 * c : kBufOOB, 0, 0, kBufNT);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // sums of x over each scale group, for this lane's rows 4 g + i
    f32x4 xs[NG];
#pragma unroll
    for (int u = 0; u < SW; ++u)
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        Acc c = {};
#pragma unroll
        for (int j = q * 4 / PER; j < (q + 1) * 4 / PER; ++j) c = Op::mul(xa[u][j], Op::ones(), c);
#pragma unroll
        for (int i = 0; i < 4; ++i) xs[u * PER + q][i] = (float)c[i];
      }
    // Tile by tile: tile t has landed once only the SW (T - 1 - t) newer
    // loads are outstanding (loads, LDS DMA included, complete in order), and
    // its products overlap the later tiles' DMA.
#pragma unroll
    for (int t = 0; t < T; ++t) {
      __builtin_amdgcn_sched_barrier(0);
      wait_newer<SW>(T - 1 - t);
      __builtin_amdgcn_sched_barrier(0);
      u32x4 cw[SW];
#pragma unroll
      for (int u = 0; u < SW; ++u) cw[u] = lds_c[wave][t][16 * nl + ((4 * u + g) ^ nl)];
#pragma unroll
      for (int u = 0; u < SW; ++u) {
        const u32x4 d = regroup<GS>(cw[u]);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
          const int at = u * PER + q;
          Acc c = {};
#pragma unroll
          for (int j = q * 4 / PER; j < (q + 1) * 4 / PER; ++j) c = Op::mul(xa[u][j], Op::unpack(d[j]), c);
          const float s = __uint_as_float(at & 1 ? sw[t][at / 2] & 0xFFFF0000u : sw[t][at / 2] << 16);
          const float z = (float)((zw[t][at / 4] >> (8 * (at & 3))) & 0xFFu);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[t][i] = __builtin_fmaf(__builtin_fmaf(-z, xs[at][i], (float)c[i]), grouped ? s * fx[at][i] : s, acc[t][i]);
        }
      }
    }
  }

  // waves are added in wave order, through the first T KB of each one's codes
  f32x4* const red_w = reinterpret_cast<f32x4*>(&lds_c[wave][0][0]);
#pragma unroll
  for (int t = 0; t < T; ++t) red_w[64 * t + lane] = acc[t];
  __syncthreads();
  for (int idx = threadIdx.x; idx < T * 64; idx += NW * 64) {
    const int t = idx >> 6, l = idx & 63;
    f32x4 sum = reinterpret_cast<const f32x4*>(&lds_c[0][0][0])[64 * t + l];
#pragma unroll
    for (int v = 1; v < NW; ++v) sum += reinterpret_cast<const f32x4*>(&lds_c[v][0][0])[64 * t + l];
    const int n = n0 + 16 * t + (l & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = 4 * (l >> 4) + i;
      if (m < M && n < N) {
        const float v = sum[i] * (kUnit<A> * (A != Act::kBf16 && !x.grouped ? x.scales[m] : 1.0f));
        if (bf16_out)
          reinterpret_cast<uint16_t*>(y)[(int64_t)m * N + n] = (uint16_t)f32_to_bf16_bits(v);
        else
          reinterpret_cast<float*>(y)[(int64_t)m * N + n] = v;
      }
    }
  }
}

#ifndef INT4_T_TALL
#define INT4_T_TALL 4
#define INT4_NW_TALL 8
#define INT4_T_SHORT 1
#define INT4_NW_SHORT 16
#endif

template <Act A>
hipError_t launch_gemv(const Int4Act& x, const Int4Weight& w, int64_t M, int64_t N, int64_t K, void* y, int b,
                       hipStream_t stream) {
  const int G = (int)((K + w.group - 1) / w.group);
  const int64_t nch = K / 32;  // 16-byte code chunks per row
  if (M == 1 && nch <= 1024) {
    const int shift = w.group == 32 ? 0 : w.group == 64 ? 1 : 2;  // chunk -> scale group
#define INT4_M1(CH, RW, S)                                                                                      \
  hipLaunchKernelGGL((int4_gemv_m1_kernel<A, CH, RW, S>), dim3((unsigned)((N + (4 / S) * RW - 1) / ((4 / S) * RW))), \
                     dim3(256), 0, stream, x, w, shift, (int)N, (int)K, G, y, b)
    if (nch <= 128) INT4_M1(1, 4, 2);         // K <= 4096
    else if (nch <= 256) INT4_M1(2, 4, 2);    // K <= 8192
    else if (nch <= 512) INT4_M1(4, 4, 2);    // K <= 16384
    else INT4_M1(4, 4, 4);                    // K <= 32768
#undef INT4_M1
    return hipGetLastError();
  }
  const int wide = K % 512 == 0 && (reinterpret_cast<uintptr_t>(w.scales) & 7) == 0 &&
                   (reinterpret_cast<uintptr_t>(w.zeros) & 3) == 0;
#define INT4_MFMA(GS, T, NW)                                                                                     \
  hipLaunchKernelGGL((int4_gemv_mfma_kernel<A, GS, T, NW>), dim3((unsigned)((N + 16 * T - 1) / (16 * T))), dim3(NW * 64), \
                     0, stream, x, w, (int)M, (int)N, (int)K, G, wide, y, b)
#define INT4_SHAPE(GS)                                           \
  if (N >= 8192) INT4_MFMA(GS, INT4_T_TALL, INT4_NW_TALL);       \
  else INT4_MFMA(GS, INT4_T_SHORT, (GS == 128 ? INT4_NW_SHORT : 8))
  if (w.group == 128) {
    INT4_SHAPE(128);
  } else if (w.group == 64) {
    INT4_SHAPE(64);
  } else {
    INT4_SHAPE(32);
  }
#undef INT4_SHAPE
#undef INT4_MFMA
  return hipGetLastError();
}

hipError_t launch_int4_gemv(const Int4Act& x, const Int4Weight& w, int64_t M, int64_t N, int64_t K, void* y,
                            bool bf16_out, hipStream_t stream) {
  const int b = bf16_out ? 1 : 0;
  if (x.type == Act::kBf16) return launch_gemv<Act::kBf16>(x, w, M, N, K, y, b, stream);
  if (x.type == Act::kI8) return launch_gemv<Act::kI8>(x, w, M, N, K, y, b, stream);
  return launch_gemv<Act::kE4m3>(x, w, M, N, K, y, b, stream);
}

}  // namespace nvfp4
