// Reductions over neighbouring lanes with DPP moves (no LDS round trip), and
// conversion to bf16 pairs, used by the group-scaled 4-bit and 8-bit kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// DPP controls (gfx9): exchanges inside 4, 8 and 16 lanes.
constexpr int kDppXor1 = 0xB1;        // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;        // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141; // lane i <-> 7 - i of 8
constexpr int kDppMirror = 0x140;     // lane i <-> 15 - i of 16

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const int64_t b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xF, 0xF, true);
  return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}

// v combined over aligned runs of L = 4, 8, 16 or 64 lanes; every lane gets
// the result.  After the exchange inside quads all four lanes agree, so the
// mirrors exchange whole quads and halves.
template <int L, class T, class F>
__device__ __forceinline__ T lanes_all(T v, F f) {
  v = f(v, dpp<kDppXor1>(v));
  v = f(v, dpp<kDppXor2>(v));
  if (L >= 8) v = f(v, dpp<kDppHalfMirror>(v));
  if (L >= 16) v = f(v, dpp<kDppMirror>(v));
  if (L >= 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}

// The same for L = 4, 8 or 16 known only at run time (uniform).
template <class T, class F>
__device__ __forceinline__ T lanes_all(T v, int L, F f) {
  v = f(v, dpp<kDppXor1>(v));
  v = f(v, dpp<kDppXor2>(v));
  if (L >= 8) v = f(v, dpp<kDppHalfMirror>(v));
  if (L >= 16) v = f(v, dpp<kDppMirror>(v));
  return v;
}

typedef __bf16 bf16_pair __attribute__((ext_vector_type(2)));
typedef float f32_pair __attribute__((ext_vector_type(2)));

// Two floats to nearest even bf16, the first in the low half (one instruction;
// the shifts and masks of f32_to_bf16_bits are five an element).
__device__ __forceinline__ uint32_t pk_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32_pair{lo, hi}), bf16_pair));
}

}  // namespace nvfp4
