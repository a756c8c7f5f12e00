// The sequence that a row of a packed batch belongs to (used by kvcache.hip;
// plain C++, so that it can be tested without a GPU).
#pragma once
#include <stdint.h>

#ifdef __HIP__
#define NVFP4_HD __host__ __device__ __forceinline__
#else
#define NVFP4_HD inline
#endif

namespace nvfp4 {

// Entries of cu that are held at hand: every cu_step(seqs)-th one and the last,
// kCuHeld + 1 in all.
constexpr int kCuHeld = 256;
NVFP4_HD int cu_step(int64_t seqs) { return (int)((seqs + kCuHeld - 1) / kCuHeld); }
NVFP4_HD int64_t cu_entry(int k, int64_t seqs) {
  const int64_t at = (int64_t)k * cu_step(seqs);
  return k == kCuHeld || at > seqs ? seqs : at;
}

// The last sequence b with cu[b] <= t < cu[b + 1], and its cu[b] as `first`; -1
// where there is none.  held[k] = cu[cu_entry(k)]; cu(i) for 0 <= i < seqs reads
// entry i, non-decreasing.  Positions are 64-bit: seqs goes up to 2^31 - 1.
template <class Held, class Cu>
NVFP4_HD int64_t sequence_of(const Held& held, const Cu& cu, int64_t seqs, int64_t t, int& first) {
  if (t < held[0] || t >= held[kCuHeld]) return -1;
  int k = 0;
#ifdef __HIP__
#pragma unroll
#endif
  for (int half = kCuHeld / 2; half > 0; half /= 2) k += held[k + half] <= t ? half : 0;  // held[k] <= t < held[k + half]
  first = held[k];
  const int step = cu_step(seqs);
  int64_t lo = (int64_t)k * step;
  if (step > 1) {
    int64_t hi = lo + step < seqs ? lo + step : seqs;
    while (hi - lo > 1) {  // cu[lo] <= t < cu[hi]
      const int64_t mid = lo + (hi - lo) / 2;
      const int v = cu(mid);
      if (v <= t) lo = mid, first = v;
      else hi = mid;
    }
  }
  return lo;
}

}  // namespace nvfp4
