// fp8_choice.h - which tile an E4M3 product with a scale per block of 128 takes,
// from its sizes alone (host code; the tests read it too).
#pragma once

#include <stdint.h>

namespace mxg {

struct F8Variant {
  int bm, bn, per_cu;
  double us, extra;
};
// the order is that of the launches in gemm_fp8.hip
constexpr F8Variant kF8Variants[] = {
    {16, 16, 2, 0.18, 1.8},   {16, 32, 2, 0.22, 1.8},   {32, 32, 1, 0.19, 2.4},   {32, 64, 2, 0.52, 1.5},
    {128, 128, 1, 0.55, 3.0}, {128, 128, 2, 1.00, 2.0}, {256, 128, 1, 0.87, 3.0}, {256, 256, 1, 1.45, 8.0}};
constexpr int kF8VariantCount = 8;

constexpr int kCus = 256;
constexpr double kBytesPerUs = 5.2e6;

// Time in us; E = 0: a dense product, else M rows over E experts.
inline double f8_estimate(const F8Variant& v, int64_t M, int64_t N, int64_t K, int64_t E) {
  // by expert the rows' split is not known here: half a tile more for each
  // expert that can have rows
  const double tiles_m = E == 0 ? (double)((M + v.bm - 1) / v.bm) : (double)M / v.bm + 0.5 * (double)(E < M ? E : M);
  const double tiles = tiles_m * (double)((N + v.bn - 1) / v.bn);
  const double full = tiles / (kCus * v.per_cu);
  const double rounds = full > 4.0 ? full + 0.5 : __builtin_ceil(full);
  const double us = v.per_cu == 2 && tiles <= kCus ? 0.7 * v.us : v.us;
  const double t = rounds * ((K + 127) / 128 * us + v.extra);
  // experts that get rows when M rows fall on E of them evenly: E M / (M + 0.6 E)
  const double used = E == 0 ? 1.0 : (double)E * M / (M + 0.6 * E);
  const double floor = used * N * K / kBytesPerUs;
  return t > floor ? t : floor;
}

// Index of the variant with the smallest estimate, the first of equal ones.
inline int f8_choice(int64_t M, int64_t N, int64_t K, int64_t E) {
  int best = 0;
  double least = f8_estimate(kF8Variants[0], M, N, K, E);
  for (int v = 1; v < kF8VariantCount; v++) {
    const double t = f8_estimate(kF8Variants[v], M, N, K, E);
    if (t < least) {
      best = v;
      least = t;
    }
  }
  return best;
}

// ---- weight gradients ---------------------------------------------------------

constexpr int kGradCus = 256;

struct GradChoice {
  bool large;
  int splits;  // of the rows; > 1: partial sums in the workspace
};
inline GradChoice grad_choice(int64_t M, int64_t N, int64_t K, int64_t E, int terms) {
  const int64_t bn = terms == 1 ? 256 : 128;
  const int64_t large = ((N + bn - 1) / bn) * ((K + 255) / 256) * E;
  if (large >= kGradCus / 2) return {true, 1};
  const int64_t small = ((N + 127) / 128) * ((K + 127) / 128) * E;
  int splits = 1;
  while (splits < 64 && small * splits * 2 <= 2 * kGradCus && M / E / (splits * 2) >= 256) splits *= 2;
  return {false, splits};
}

}  // namespace mxg
