// Which kernels take an FP8 product (used by fp8_gemm.hip; plain C++, so that it
// can be tested without a GPU).
#pragma once
#include <stdint.h>

namespace nvfp4 {

// Few rows (rows and columns of 16 a workgroup, waves); many rows (rows and columns a workgroup).
enum Fp8Kernel {
  kNoKernel,
  kRows1x1,
  kRows1x2,
  kRows2x1,
  kRows2x2Of8,
  kRows2x2Of4,
  kTile32x64,
  kTile64x64,
  kTile64x128,
  kTile128x128,
  kTile128x256,
  kTile256x256
};

// `first` takes the first M rows and N columns of a product, `second` the other
// columns, or the other rows (kNoKernel: there are none).
struct Fp8Plan {
  Fp8Kernel first, second;
  int64_t M, N;
};

// Kernels of many rows, and the time of a step (a block of 128 columns of all
// tiles) of theirs in us: that of the rounds of workgroups that the 256 CUs take,
// one a CU, or where `both` is given two.  Of 333 sizes (M = 32 .. 8192, N = 1024, 4096,
// 5000, 14336, K = 1024, 4096, 14336, either output) the choice was within 8% of the
// fastest kernel in 318 and within 15% in 329; in the other four, up to 31% slower
// (2048 x 5000 x 14336 to fp32 400 us, with 128 x 128 tiles 306), half or less of a last
// round of two a CU counts as a full one.  us at K = 4096 in the order below, to bf16:
// 128 x 4096 12.3 / 11.8 / 15.5 / 20.9 / 29.0 / 41.3; 256 x 4096 14.5 / 12.2 / 15.7 / 21.0 /
// 29.1 / 43.6; 512 x 14336 98 / 70 / 57 / 42.8 / 36.7 / 51.0; 1024 x 4096 52 / 35.3 / 26.5 /
// 23.5 / 31.6 / 45.5; 4096 x 4096 208 / 129 / 103 / 76 / 74 / 61.1; to fp32: 512 x 4096 26.6 /
// 24.1 / 35.3; 2048 x 4096 96.8 / 76.9 / 65.7.  (From K = 4096 to 14336 a step of a full
// round takes 0.3 / 0.35 / 0.54 / 0.66 / 1.0 / 1.7, to fp32 0.48 / 0.7 / 1.08.)
struct Fp8Tiles {
  Fp8Kernel kernel;
  int bm, bn;
  double alone, both;
  int64_t tiles_m(int64_t M) const { return (M + bm - 1) / bm; }
  int64_t tiles_n(int64_t N) const { return (N + bn - 1) / bn; }
  double step(int64_t M, int64_t N) const {
    const int64_t t = tiles_m(M) * tiles_n(N);
    return both > 0 && t > 256 ? (double)((t + 511) / 512) * both : (double)((t + 255) / 256) * alone;
  }
};
constexpr Fp8Tiles kFp8Tiles16[] = {{kTile32x64, 32, 64, 0.30, 0.46},    {kTile64x64, 64, 64, 0.33, 0.64},
                                    {kTile64x128, 64, 128, 0.50, 0.88},  {kTile128x128, 128, 128, 0.66, 1.15},
                                    {kTile128x256, 128, 256, 1.07, 0.0}, {kTile256x256, 256, 256, 1.80, 0.0}};
constexpr Fp8Tiles kFp8Tiles32[] = {
    {kTile64x64, 64, 64, 0.47, 0.78}, {kTile64x128, 64, 128, 0.73, 1.30}, {kTile128x128, 128, 128, 1.15, 2.00}};
// The last one's conditions: two pairs of steps at least, and rows of y that 32-bit offsets reach.
inline bool fp8_can_256(int64_t N, int64_t K) { return K > 256 && N <= (int64_t)1 << 21; }

// The kernel of the least estimated time, or two: whole rounds of one with one
// workgroup a CU for the first columns or rows and the best for the rest, where
// that looks 5% better or more (1000 x 20000 x 4096: 1.2 rounds of 256 x 256 tiles
// 119 us, one round and one of 128 x 128 88; 6000 x 4096 x 4096 107 and 99; 4096 x
// 14336 x 4096, 3.5 rounds, 226 and 224: the clock is at its power limit. Two
// workgroups a CU do not end together: 2048 x 14336 x 4096 to fp32 245 and 255).
inline Fp8Plan fp8_plan_tiles(int64_t M, int64_t N, int64_t K, bool bf16) {
  const Fp8Tiles* all = bf16 ? kFp8Tiles16 : kFp8Tiles32;
  const int n = !bf16 ? 3 : fp8_can_256(N, K) ? 6 : 5;
  const auto best = [&](int64_t m, int64_t c, double& us) {
    const Fp8Tiles* b = all;
    us = b->step(m, c);
    for (int i = 1; i < n; ++i)
      if (const double t = all[i].step(m, c); t < us) us = t, b = all + i;
    return b->kernel;
  };
  double us;
  Fp8Plan plan{best(M, N, us), kNoKernel, M, N};
  const double apart = 3.0 * 128 / (double)K;  // of a second launch
  us *= 0.95;
  for (int i = 0; i < n; ++i) {
    const Fp8Tiles& k = all[i];
    const int64_t tm = k.tiles_m(M), tn = k.tiles_n(N), whole = tm * tn / 256 * 256;
    if (k.both > 0 || whole == 0) continue;
    const auto consider = [&](int64_t m, int64_t c, int64_t m2, int64_t c2) {
      if (m == 0 || c == 0 || m2 <= 0 || c2 <= 0) return;
      double rest;
      const Fp8Kernel b = best(m2, c2, rest);
      if (const double t = k.step(m, c) + rest + apart; t < us) us = t, plan = {k.kernel, b, m, c};
    };
    consider(M, whole / tm * k.bn, M, N - whole / tm * k.bn);  // (bn is a multiple of 128)
    consider(whole / tn * k.bm, N, M - whole / tn * k.bm, N);
  }
  return plan;
}

// Few rows in all: workgroups of few waves that share nothing but their sums,
// as long as there are about two of them a CU at most; from there on tiles
// through LDS, by their estimated time.
// (us, K = 4096: M = 16, N = 1024 / 4096 / 14336: rows<1, 1> 4.6 / 6.4 / 17.0, rows<1, 2> 5.7 / 7.5 (8 waves), - / - / 14.6
// (4); M = 32, N = 4096: rows<2, 1> 7.8, rows<2, 2> 9.9; M = 64, N = 4096: rows<2, 2> of 8 waves 9.8, 32 x 64 tiles 12.2; M =
// 128, N = 4096: rows<2, 2> of 4 waves 14.3, 32 x 64 tiles 12.6, to fp32 14.3 and 18.9, 64 x 64 tiles 18.1.)
inline Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t K, bool bf16) {
  const auto tiles = [&](int64_t bm, int64_t bn) { return (M + bm - 1) / bm * ((N + bn - 1) / bn); };
  if (M <= 16) return {tiles(16, 16) <= 512 ? kRows1x1 : kRows1x2, kNoKernel, M, N};
  const int64_t t = tiles(32, 16);
  if (t <= 256) return {kRows2x1, kNoKernel, M, N};
  if (t <= 512) return {kRows2x2Of8, kNoKernel, M, N};
  if (!bf16 && t <= 1024) return {kRows2x2Of4, kNoKernel, M, N};
  return fp8_plan_tiles(M, N, K, bf16);
}

}  // namespace nvfp4
