// Decode products y = x W^T for group-scaled 4-bit integer weights and bf16,
// INT8 or E4M3 activations, M <= 16 rows (format: include/int4.h):
//   y[m, n] = sum_g s[n, g] sx[m, g] (sum_{k in g} x c - z[n, g] sum_{k in g} x)
// The codes c = 0..15 go into the products as they are: a mask and a shift
// turn 8 nibbles into 8 bytes, and such a byte is at once the INT8 value c
// and the E4M3 value c / 512 (subnormals and the first binade are evenly
// spaced).  INT8 activations meet them in integer products (exact inside a
// group); for bf16 and E4M3 ones the FP8 converter, which multiplies by a
// power of two on the way, makes exact bf16 pairs c.  The zero point is taken
// off with the sum of x, which all rows of the weight share.
#include "device_common.hpp"
#include "int4_kernels.hpp"

namespace nvfp4 {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kPassSupers = 4;  // super-chunks of 128 codes a pass of the matrix kernel takes

constexpr uint32_t kNibbles = 0x0F0F0F0Fu;

// ---- one row (M = 1): dot products on the vector units.
// A workgroup of 4 waves: S waves split K, the 4 / S wave groups take RW rows
// each.  Lane l of a wave has the 16-byte chunks (32 codes, inside one group)
// l, l + 64, ... of its K part, so one load instruction reads 1 KB of a row,
// and keeps the x of its chunks and their sums in registers for all its rows.
// Loads past the K part, or of rows past N, return zeros.  Bound by latency at
// the sizes that come here: 1024 x 4096, INT8, 3.3 us (2.2 MB), where an empty
// kernel takes 2.5.
template <Act A>
struct Chunk {             // x of one chunk
  uint32_t x[A == Act::kI8 ? 8 : 16];
  float sum;
  float scale;
};

__device__ __forceinline__ float dot2_bf16(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
}
// Two E4M3 bytes (the low or the high half of w) as a bf16 pair, and two codes.
__device__ __forceinline__ uint32_t pk_bf16_e4m3(uint32_t w, bool high) {
  return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                                           : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}
__device__ __forceinline__ uint32_t pk_bf16_code(uint32_t w, bool high) {
  return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.0f, true)
                                           : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.0f, false));
}
constexpr uint32_t kOnes = 0x3F803F80u;  // a bf16 pair

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
      s = dot2_bf16(c.x[j], kOnes, s);
    }
    c.sum = s;
  }
}

// sum over a chunk of x (code - z)
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
      p[d & 1] = dot2_bf16(c.x[4 * d], pk_bf16_code(lo, false), p[d & 1]);
      p[d & 1] = dot2_bf16(c.x[4 * d + 1], pk_bf16_code(lo, true), p[d & 1]);
      p[d & 1] = dot2_bf16(c.x[4 * d + 2], pk_bf16_code(hi, false), p[d & 1]);
      p[d & 1] = dot2_bf16(c.x[4 * d + 3], pk_bf16_code(hi, true), p[d & 1]);
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
  const __amdgpu_buffer_rsrc_t zbuf = make_buf(w.zeros ? w.zeros + rb * G : nullptr,
                                               w.zeros ? (uint32_t)(nrows * G) : 0u);
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
    for (int c = 0; c < CH; ++c) {
      const float d = dot_chunk<A>(xc[c], cw[r][c], (float)zw[r][c]), s = bf16_bits_to_f32(sw[r][c]);
      acc[r] = A == Act::kBf16 ? __builtin_fmaf(d, s, acc[r]) : __builtin_fmaf(d * s, xc[c].scale, acc[r]);
    }
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
    if (A != Act::kBf16 && !x.grouped) sum *= x.scales[0];
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
// DMA, every instruction reading 4 rows x 256 contiguous bytes, the 16-byte
// chunks of a row swizzled so that no read back has bank conflicts.  A matrix
// instruction adds up over the lane groups g (lane = 16 g + n, n a row of the
// weight), and which 8 of the 128 codes each group feeds it is free as long as
// x agrees and all 32 belong to one scale group: two dwords each of half a
// super-chunk for two instructions (one 8-byte read; 16 bytes of 8-bit x serve
// both), or, for groups of 32, one dword each of a chunk.
//
// Reading x costs as much as reading the codes: every workgroup reads all of
// it, from L2, and a load instruction takes the same 16 cycles of the address
// path whether its lanes are live or not.  So x is read like the codes, 4
// rows x 256 contiguous bytes an instruction and none for rows past M, and
// put into the operands' layout through LDS.  (Loads straight into that
// layout, 16 rows x 64 bytes, meet on few L2 channels where K is a large power
// of two: 14336 x 4096 at M = 16, bf16, took 11.6 us instead of 10.6.)  So are
// the scales, which the four lane groups would otherwise each load (8.5 us
// instead of 9.0 on that weight at M = 1).
//
// A product of one scale group starts at zero, the zero point is taken off with
// the sum of x over the group (a matrix product with a constant operand, shared
// by the T row tiles), and the difference is added into the fp32 sums with its
// scale.  The difference has to be formed inside the group, where INT8 sums are
// whole numbers: s z sum x of several groups as one fp32 matrix product saves
// the multiply-adds (4096 x 14336, M = 1, bf16: 8.7 us instead of 8.9; INT8 7.1,
// 7.2; M = 16 13.1, 13.0) but makes the fp32 sums as large as the code part of
// a pass (14336 x 4096, M = 16, x of one sign: relative error 2.3e-6 for bf16
// and 1.2e-6 for INT8 instead of 3.4e-8 and 2.5e-8).
//
// Bound: memory and, right behind it, vector issue.  14336 x 4096, bf16, M = 1:
// 30.8 MB in 8.4 us a call from memory (3.7 TB/s; 8.0 from the last-level cache,
// where the DMA alone, with nothing computed, takes 6.5-6.9); about 910 vector
// instructions a wave are 3.0 us of issue, half of them unpacking codes.  INT8
// unpacks in 3 instructions for 8 codes instead of 7 and takes 7.7 us; M = 16:
// INT8 9.1, E4M3 with grouped scales 9.9, bf16 10.1 us.  4096 x 14336, bf16: M = 1
// 10.8, M = 16 13.9 us (9.4 and 13.3 from the cache); a workgroup takes 7 us even
// where only a quarter of the CUs have one, reading x among it.
//
// E4M3 activations are widened to bf16 as well: the FP8 matrix instruction
// keeps too few bits of its sums (9e-5 off, relative, after 160 products,
// where the bf16 one is off by less than 1e-6).
template <Act A>
struct Mfma {
  using Acc = f32x4;
  using X = u32x4;   // 8 bf16
  static __device__ __forceinline__ Acc mul(X x, X w, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, w), c, 0,
                                                   0, 0);
  }
  static __device__ __forceinline__ X unpack(uint32_t w) {
    const uint32_t lo = w & kNibbles, hi = (w >> 4) & kNibbles;
    return X{pk_bf16_code(lo, false), pk_bf16_code(lo, true), pk_bf16_code(hi, false), pk_bf16_code(hi, true)};
  }
  static __device__ __forceinline__ X of(u32x2 v) {  // 8 E4M3 activations
    return X{pk_bf16_e4m3(v.x, false), pk_bf16_e4m3(v.x, true), pk_bf16_e4m3(v.y, false), pk_bf16_e4m3(v.y, true)};
  }
  static __device__ __forceinline__ X ones() { return X{kOnes, kOnes, kOnes, kOnes}; }
};
template <>
struct Mfma<Act::kI8> {
  using Acc = i32x4;
  using X = u32x2;
  static __device__ __forceinline__ Acc mul(X x, X w, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, x), __builtin_bit_cast(long, w), c, 0, 0, 0);
  }
  static __device__ __forceinline__ X unpack(uint32_t w) { return X{w & kNibbles, (w >> 4) & kNibbles}; }
  static __device__ __forceinline__ X of(u32x2 v) { return v; }
  static __device__ __forceinline__ X ones() { return X{0x01010101u, 0x01010101u}; }
};

// LDS written by other lanes of the wave is read after this (a wave's LDS
// operations complete in order: only the compiler has to keep it).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// What a wave loads into registers for one pass; all of it goes through LDS
// to the lanes that need it (loads in the operands' layout would be more
// instructions of fewer live lanes each).
template <Act A, bool GX, int GS, int T, int MQ>
struct Pass {
  static constexpr int XB = A == Act::kBf16 ? 2 : 1;  // bytes of an activation
  static constexpr int XR = 2 * XB;                   // rounds of 16 rows x 256 bytes that x goes through LDS in
  static constexpr int NG = kPassSupers * 128 / GS;   // scale groups
  static constexpr int SI = (16 * T * NG / 4 + 63) / 64;
  u32x4 x[XR][MQ];   // x: 4 MQ rows
  u32x2 s[SI];       // scales of 4 groups of a row: item i = 64 a + lane is row i % 16T, groups 4 (i / 16T)..
  uint32_t z[SI];    // and their zero points
  float f[GX ? NG / 4 : 1];  // grouped scales of x: row lane % 16, group 4 a + lane / 16
};

// GX: x has a scale for each group.  MQ: 4 MQ rows of x are read (M <= 4 MQ).
template <Act A, bool GX, int GS, int T, int NW, int MQ>
__global__ __launch_bounds__(NW * 64) void int4_gemv_mfma_kernel(Int4Act x, Int4Weight w, int M, int N, int K, int G,
                                                                 int wide, void* __restrict__ y, int bf16_out) {
  using Op = Mfma<A>;
  using Acc = typename Op::Acc;
  using P = Pass<A, GX, GS, T, MQ>;
  constexpr int SW = kPassSupers, XB = P::XB, XR = P::XR, NG = P::NG;
  constexpr int PER = 128 / GS;                       // scale groups of a super-chunk
  constexpr bool PAIRS = GS >= 64;
  constexpr int R = 16 * T;                           // rows of the workgroup
  static_assert(T <= 4, "one LDS array per tile");
  // One array per row tile: the compiler then knows which DMA a read depends
  // on and waits for that one only (with one array for all tiles the first
  // tile's reads waited for every DMA in flight: 14336 x 4096, M = 16, INT8,
  // 9.8 us instead of 9.2).
  __shared__ u32x4 lds_c0[NW][256], lds_c1[NW][256], lds_c2[NW][256], lds_c3[NW][256];
  __shared__ u32x4 lds_x[NW][256];
  __shared__ __align__(16) uint32_t lds_s[NW][T == 1 ? (GX ? 28 : 12) * NG : 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const auto tile = [&](int t) {  // t is a constant once the loops are unrolled
    return t == 0 ? lds_c0[wave] : t == 1 ? lds_c1[wave] : t == 2 ? lds_c2[wave] : lds_c3[wave];
  };
  // Scales [NG / 4][R] pairs of dwords, zero points [NG / 4][R], grouped scales
  // of x [NG][16]; with several tiles in the place of x, which is in registers
  // by then.
  uint32_t* const st_s = T == 1 ? lds_s[wave] : reinterpret_cast<uint32_t*>(lds_x[wave]);
  uint32_t* const st_z = st_s + R * NG / 2;
  float* const st_f = reinterpret_cast<float*>(st_z + R * NG / 4);
  static_assert(T == 1 || (R * NG * 3 / 4 + 16 * NG) * 4 <= 4096, "scales fit the place of x");
  const int nl = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * (16 * T);
  const int rows = min(R, N - n0);
  const int half = K / 2;
  const __amdgpu_buffer_rsrc_t cbuf = make_buf(w.codes + (int64_t)n0 * half, (uint32_t)(rows * half));
  const __amdgpu_buffer_rsrc_t sbuf = make_buf(w.scales + (int64_t)n0 * G, (uint32_t)(rows * G * 2));
  const __amdgpu_buffer_rsrc_t zbuf = make_buf(w.zeros ? w.zeros + (int64_t)n0 * G : nullptr,
                                               w.zeros ? (uint32_t)(rows * G) : 0u);
  const __amdgpu_buffer_rsrc_t xbuf = make_buf(x.x, (uint32_t)(M * K * XB));
  const __amdgpu_buffer_rsrc_t fbuf = make_buf(x.scales, GX ? (uint32_t)(M * G * 4) : 0u);
  const int nch = K / 32, nsc = (nch + 3) / 4;
  const int per = ((nsc + NW - 1) / NW + SW - 1) / SW * SW;  // whole passes, so scales are read in aligned runs
  const int sbeg = wave * per, send = min(sbeg + per, nsc);

  f32x4 acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Byte offsets of this lane's loads at super-chunk 0.
  int x_at[MQ], c_at[SW];
#pragma unroll
  for (int q = 0; q < MQ; ++q) {
    const int row = 4 * q + g;
    x_at[q] = row < M ? row * K * XB + 16 * nl : kBufOOB;
  }
#pragma unroll
  for (int u = 0; u < SW; ++u) {
    const int r = 4 * u + g;
    c_at[u] = r * half + 16 * (nl ^ r);
  }
  const auto dma = [&](int t, int u, int off) {
    // non-temporal: each code byte is read once
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        cbuf, (__attribute__((address_space(3))) void*)(tile(t) + 64 * u), 16, off, 0, 0, kBufNT);
  };
  // The loads of the pass from super-chunk s0: x (L2 hits), then scales, then
  // codes, so that what comes first is waited for first.  x comes 4 rows x 256
  // contiguous bytes an instruction; DMA instruction u of tile t fills LDS
  // slots [64 u, 64 u + 64): lane l -> row r = 4 u + l / 16, slot j = l % 16,
  // holding chunk 4 s0 + (j ^ r).
  const auto load = [&](P& p, int s0) {
    const int g0 = s0 * PER;  // first scale group of the pass
    if (wide && s0 + SW <= send) {
      // K % 512 == 0 and aligned pointers: the whole pass lies inside the rows
#pragma unroll
      for (int v = 0; v < XR; ++v)
#pragma unroll
        for (int q = 0; q < MQ; ++q)
          p.x[v][q] = __builtin_amdgcn_raw_buffer_load_b128(xbuf, x_at[q] + 128 * XB * s0, 256 * v, 0);
#pragma unroll
      for (int a = 0; a < P::SI; ++a) {
        const int item = 64 * a + lane;
        const int base = R * NG / 4 % 64 == 0 || item < R * NG / 4 ? item % R * G + g0 + 4 * (item / R) : kBufOOB / 2;
        p.s[a] = __builtin_amdgcn_raw_buffer_load_b64(sbuf, 2 * base, 0, 0);
        p.z[a] = w.zeros ? __builtin_amdgcn_raw_buffer_load_b32(zbuf, base, 0, 0) : 0x08080808u;
      }
      if constexpr (GX) {
#pragma unroll
        for (int a = 0; a < NG / 4; ++a)
          p.f[a] = __builtin_bit_cast(
              float, __builtin_amdgcn_raw_buffer_load_b32(fbuf, 4 * (nl * G + g0 + 4 * a + g), 0, 0));
      }
#pragma unroll
      for (int t = 0; t < T; ++t) {
        __builtin_amdgcn_sched_barrier(0);  // tile order
#pragma unroll
        for (int u = 0; u < SW; ++u) dma(t, u, c_at[u] + 16 * t * half + 64 * s0);
      }
    } else {
      // any K: what lies past K or this wave's range reads as zero
      const int kend = min(K, 128 * send);
#pragma unroll
      for (int v = 0; v < XR; ++v)
#pragma unroll
        for (int q = 0; q < MQ; ++q) {
          const int k = 128 * s0 + (256 * v + 16 * nl) / XB;
          p.x[v][q] = __builtin_amdgcn_raw_buffer_load_b128(
              xbuf, k < kend ? x_at[q] + 128 * XB * s0 + 256 * v : kBufOOB, 0, 0);
        }
#pragma unroll
      for (int a = 0; a < P::SI; ++a) {
        const int item = 64 * a + lane, row = item % R, gq = g0 + 4 * (item / R);
        uint32_t s[4], z = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int at = item < R * NG / 4 && gq + q < G ? row * G + gq + q : kBufOOB / 2;
          s[q] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(sbuf, 2 * at, 0, 0) & 0xFFFFu;
          z |= (w.zeros ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(zbuf, at, 0, 0) & 0xFFu : 8u) << (8 * q);
        }
        p.s[a] = u32x2{s[0] | (s[1] << 16), s[2] | (s[3] << 16)};
        p.z[a] = z;
      }
      if constexpr (GX) {
#pragma unroll
        for (int a = 0; a < NG / 4; ++a) {
          const int q = g0 + 4 * a + g;
          p.f[a] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                 fbuf, q < G ? 4 * (nl * G + q) : kBufOOB, 0, 0));
        }
      }
#pragma unroll
      for (int t = 0; t < T; ++t) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < SW; ++u)
          dma(t, u, 4 * s0 + (nl ^ (4 * u + g)) < min(nch, 4 * send) ? c_at[u] + 16 * t * half + 64 * s0 : kBufOOB);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // x of round v through LDS into the operands' layout: piece p (16 bytes) of
  // row r lies in slot p ^ r of the row, so neither side has bank conflicts.
  // Rows past 4 MQ are not written; what is read there only reaches sums of
  // rows past M.  Fills xa for the round's super-chunks and xs with the sums of
  // x over their scale groups, for row nl of x.
  const auto spread = [&](const P& p, int v, typename Op::X (&xa)[SW][4]) {
    wave_fence();
#pragma unroll
    for (int q = 0; q < MQ; ++q) {
      const int row = 4 * q + (lane >> 4);
      lds_x[wave][16 * row + ((lane & 15) ^ row)] = p.x[v][q];
    }
    wave_fence();
    const u32x4* const xrow = &lds_x[wave][16 * nl];
#pragma unroll
    for (int u = v * SW / XR; u < (v + 1) * SW / XR; ++u) {
      const int p0 = 8 * XB * (u - v * SW / XR);  // first piece of super-chunk u
#pragma unroll
      for (int j = 0; j < 4; j += PAIRS && XB == 1 ? 2 : 1) {
        if constexpr (A == Act::kBf16) {
          xa[u][j] = xrow[(p0 + (PAIRS ? 4 * (j & 2) + 2 * g + (j & 1) : 4 * j + g)) ^ nl];
        } else if constexpr (PAIRS) {
          const u32x4 d = xrow[(p0 + 2 * j + g) ^ nl];
          xa[u][j] = Op::of(u32x2{d.x, d.y});
          xa[u][j + 1] = Op::of(u32x2{d.z, d.w});
        } else {
          xa[u][j] = Op::of(reinterpret_cast<const u32x2*>(&xrow[(p0 + 2 * j + (g >> 1)) ^ nl])[g & 1]);
        }
      }
    }
  };

  // Sums of x over the scale groups of super-chunk u, for the four rows of x
  // that this lane has in an accumulator.
  const auto sums_of = [&](int u, const typename Op::X (&xa)[SW][4], f32x4 (&xs)[NG]) {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      Acc c = {};
#pragma unroll
      for (int j = q * 4 / PER; j < (q + 1) * 4 / PER; ++j) c = Op::mul(xa[u][j], Op::ones(), c);
#pragma unroll
      for (int i = 0; i < 4; ++i) xs[u * PER + q][i] = (float)c[i];
    }
  };

  // The dwords of codes this lane feeds to the four matrix instructions of
  // super-chunk u: in pairs, instruction j takes dword 2 (g & 1) + j % 2 of
  // chunk 2 (j / 2) + g / 2; otherwise dword g of chunk j.
  // (Byte 256 n + 16 (chunk ^ n) + 4 dword of the tile: u and j are constants,
  // so an address is one exclusive or; made anew for every pass, since kept
  // they would cost 16 registers.)
  int code_at = PAIRS ? 256 * nl + 16 * (nl ^ (g >> 1)) + 8 * (g & 1) : 272 * nl + 4 * g;
  const auto codes_of = [&](int t, int u) {
    const char* const codes = reinterpret_cast<const char*>(tile(t));
    u32x4 d;
#pragma unroll
    for (int j = 0; j < 4; j += PAIRS ? 2 : 1) {
      const char* const at = codes + (code_at ^ (64 * u + 16 * j));
      if constexpr (PAIRS) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(at);
        d[j] = v.x;
        d[j + 1] = v.y;
      } else {
        d[j] = *reinterpret_cast<const uint32_t*>(at);
      }
    }
    return d;
  };

  // Scales, zero points and grouped scales of x to LDS.
  const auto spread_scales = [&](const P& p) {
    wave_fence();
#pragma unroll
    for (int a = 0; a < P::SI; ++a) {
      const int item = 64 * a + lane;
      if (R * NG / 4 % 64 == 0 || item < R * NG / 4) {
        reinterpret_cast<u32x2*>(st_s)[item] = p.s[a];
        st_z[item] = p.z[a];
      }
    }
    if constexpr (GX) {
#pragma unroll
      for (int a = 0; a < NG / 4; ++a) st_f[64 * a + lane] = p.f[a];  // [group 4 a + g][row nl]
    }
    wave_fence();
  };

  // Products of super-chunk u of tile t.
  const auto multiply = [&](int t, int u, u32x4 w4, const typename Op::X (&xa)[SW][4], const f32x4 (&xs)[NG]) {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int at = u * PER + q;
      const u32x2 s4 = reinterpret_cast<const u32x2*>(st_s)[at / 4 * R + 16 * t + nl];
      const uint32_t z4 = st_z[at / 4 * R + 16 * t + nl];
      Acc c = {};
#pragma unroll
      for (int j = q * 4 / PER; j < (q + 1) * 4 / PER; ++j) c = Op::mul(xa[u][j], Op::unpack(w4[j]), c);
      const uint32_t s2 = at & 2 ? s4.y : s4.x;
      const float s = __uint_as_float(at & 1 ? s2 & 0xFFFF0000u : s2 << 16);
      const float z = (float)((z4 >> (8 * (at & 3))) & 0xFFu);
      // (d s) sx and not d (s sx): the product of the scales may leave fp32's
      // range where the result does not
      f32x4 sx;
      if constexpr (GX) sx = *reinterpret_cast<const f32x4*>(&st_f[16 * at + 4 * g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float d = __builtin_fmaf(-z, xs[at][i], (float)c[i]);
        acc[t][i] = GX ? __builtin_fmaf(d * s, sx[i], acc[t][i]) : __builtin_fmaf(d, s, acc[t][i]);
      }
    }
  };

  const auto compute = [&](const P& p) {
    typename Op::X xa[SW][4];
    f32x4 xs[NG];
    if constexpr (T == 1) {
      // round by round: few operands are live
      spread_scales(p);
#pragma unroll
      for (int v = 0; v < XR; ++v) {
        spread(p, v, xa);
#pragma unroll
        for (int u = v * SW / XR; u < (v + 1) * SW / XR; ++u) {
          sums_of(u, xa, xs);
          multiply(0, u, codes_of(0, u), xa, xs);
        }
      }
    } else {
      // tile by tile, in the order of the DMA, so that a tile's products
      // overlap the later tiles' DMA
#pragma unroll
      for (int v = 0; v < XR; ++v) spread(p, v, xa);
#pragma unroll
      for (int u = 0; u < SW; ++u) sums_of(u, xa, xs);
      spread_scales(p);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        __builtin_amdgcn_sched_barrier(0);
        u32x4 cw[SW];
#pragma unroll
        for (int u = 0; u < SW; ++u) cw[u] = codes_of(t, u);
#pragma unroll
        for (int u = 0; u < SW; ++u) multiply(t, u, cw[u], xa, xs);
      }
    }
  };

  for (int s0 = sbeg; s0 < send; s0 += SW) {  // wave-uniform
    asm volatile("" : "+v"(code_at));
    P p;
    load(p, s0);
    compute(p);
  }

  // waves are added in wave order, through each one's first tile of codes
  f32x4* const red_w = reinterpret_cast<f32x4*>(lds_c0[wave]);
#pragma unroll
  for (int t = 0; t < T; ++t) red_w[64 * t + lane] = acc[t];
  __syncthreads();
  for (int idx = threadIdx.x; idx < T * 64; idx += NW * 64) {
    const int t = idx >> 6, l = idx & 63;
    f32x4 sum = reinterpret_cast<const f32x4*>(lds_c0[0])[64 * t + l];
#pragma unroll
    for (int v = 1; v < NW; ++v) sum += reinterpret_cast<const f32x4*>(lds_c0[v])[64 * t + l];
    const int n = n0 + 16 * t + (l & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = 4 * (l >> 4) + i;
      if (m < M && n < N) {
        const float v = A != Act::kBf16 && !GX ? sum[i] * x.scales[m] : sum[i];
        if (bf16_out)
          reinterpret_cast<uint16_t*>(y)[(int64_t)m * N + n] = (uint16_t)f32_to_bf16_bits(v);
        else
          reinterpret_cast<float*>(y)[(int64_t)m * N + n] = v;
      }
    }
  }
}

// Waves and rows per workgroup, from a sweep over 16 and 32 and 64 rows at the
// sizes named here, M = 1 and 16, all types, groups of 128 (us a call, queued
// back to back, the weights from memory):
//  * N <= 4096: 16 rows, so that up to 256 CUs have a workgroup each; 16 waves
//    where K has more than one pass for each of 8 (4096 x 14336, bf16, M =
//    16: 14.2 with 16, 14.9 with 8; M = 1: 9.5, 10.1; 4096 x 4096: 6.4, 6.3);
//    just above that length 8 waves are still as good (4096 x 8192, M = 1: 7.7
//    with 16, 7.2 with 8);
//  * N <= 8192: 32 rows for the same reason (8192 x 4096, INT8, M = 16: 6.8;
//    16 rows 7.2, 64 rows 7.8; 5120 x 5120, bf16, M = 16: 8.4, 10.7, 11.7);
//  * above: 64 rows, x being read once per workgroup (14336 x 4096, INT8, M =
//    16: 9.1; 32 rows 11.3, 16 rows 12.3; 28672 x 4096, bf16, M = 1: 15.1, 17.6,
//    16.6).
// A workgroup of 64 rows fills a CU's LDS, so N a little above 16384 takes a
// second, nearly empty round: there 16 rows are faster at M = 1 (17408 x 5120,
// bf16: 15.6 instead of 19.7; 18944 x 3584: 11.6, 13.4) and no shape gains at M
// = 16 (22.1 against 21.5 and 22.2; 15.9 and 16.0).
//
// x of 5 to 8 rows is read as 8 rows, not 16: 14336 x 4096, M = 5, bf16 8.6 us
// instead of 9.1, INT8 8.0, 8.2; 4096 x 14336, M = 8, bf16 10.8, 12.0; 28672 x
// 8192, M = 5, bf16 31.2, 32.6 (the weights of the first two from the last-level
// cache).
template <Act A, bool GX>
hipError_t launch_mfma(const Int4Act& x, const Int4Weight& w, int64_t M, int64_t N, int64_t K, int G, void* y, int b,
                       hipStream_t stream) {
  const int wide = K % 512 == 0 && (reinterpret_cast<uintptr_t>(w.scales) & 7) == 0 &&
                   (reinterpret_cast<uintptr_t>(w.zeros) & 3) == 0;
#define INT4_MFMA(GS, T, NW, MQ)                                                                                   \
  hipLaunchKernelGGL((int4_gemv_mfma_kernel<A, GX, GS, T, NW, MQ>), dim3((unsigned)((N + 16 * T - 1) / (16 * T))), \
                     dim3(NW * 64), 0, stream, x, w, (int)M, (int)N, (int)K, G, wide, y, b)
#define INT4_ROWS(GS, T, NW)                  \
  do {                                        \
    if (M <= 4) INT4_MFMA(GS, T, NW, 1);      \
    else if (M <= 8) INT4_MFMA(GS, T, NW, 2); \
    else INT4_MFMA(GS, T, NW, 4);             \
  } while (0)
#define INT4_SHAPE(GS)                          \
  do {                                          \
    if (N > 8192) INT4_ROWS(GS, 4, 8);          \
    else if (N > 4096) INT4_ROWS(GS, 2, 8);     \
    else if (K > 4096) INT4_ROWS(GS, 1, 16);    \
    else INT4_ROWS(GS, 1, 8);                   \
  } while (0)
  if (w.group == 128) INT4_SHAPE(128);
  else if (w.group == 64) INT4_SHAPE(64);
  else INT4_SHAPE(32);
#undef INT4_SHAPE
#undef INT4_ROWS
#undef INT4_MFMA
  return hipGetLastError();
}

// One row of few weights goes to the dot products, which start sooner (bf16, us
// a call with the weights from memory: 1024 x 4096 3.4, the matrix kernel 4.2;
// 1024 x 14336 5.9, 7.8; 4096 x 4096 4.8, 5.0; 4096 x 8192 6.6, 7.1); a large weight
// to the matrix kernel, which reads longer runs (4096 x 14336: 11.7, 10.5; 14336
// x 4096: 9.2, 8.4; 8192 x 4096: 6.3, 6.0).  K is split over 2 or 4 waves.
template <Act A>
hipError_t launch_gemv(const Int4Act& x, const Int4Weight& w, int64_t M, int64_t N, int64_t K, void* y, int b,
                       hipStream_t stream) {
  const int G = (int)((K + w.group - 1) / w.group);
  if (M == 1 && K <= 16384 && (N <= 2048 || (N <= 4096 && K <= 8192))) {
    const int shift = w.group == 32 ? 0 : w.group == 64 ? 1 : 2;  // chunk -> scale group
#define INT4_M1(CH, RW, S)                                                                                           \
  hipLaunchKernelGGL((int4_gemv_m1_kernel<A, CH, RW, S>), dim3((unsigned)((N + (4 / S) * RW - 1) / ((4 / S) * RW))), \
                     dim3(256), 0, stream, x, w, shift, (int)N, (int)K, G, y, b)
    if (K <= 4096) INT4_M1(1, 2, 2);       // CH S 64 chunks of 32
    else if (K <= 8192) INT4_M1(1, 2, 4);
    else INT4_M1(2, 2, 4);
#undef INT4_M1
    return hipGetLastError();
  }
  if constexpr (A != Act::kBf16) {
    if (x.grouped) return launch_mfma<A, true>(x, w, M, N, K, G, y, b, stream);
  }
  return launch_mfma<A, false>(x, w, M, N, K, G, y, b, stream);
}

hipError_t launch_int4_gemv(const Int4Act& x, const Int4Weight& w, int64_t M, int64_t N, int64_t K, void* y,
                            bool bf16_out, hipStream_t stream) {
  const int b = bf16_out ? 1 : 0;
  if (x.type == Act::kBf16) return launch_gemv<Act::kBf16>(x, w, M, N, K, y, b, stream);
  if (x.type == Act::kI8) return launch_gemv<Act::kI8>(x, w, M, N, K, y, b, stream);
  return launch_gemv<Act::kE4m3>(x, w, M, N, K, y, b, stream);
}

}  // namespace nvfp4
