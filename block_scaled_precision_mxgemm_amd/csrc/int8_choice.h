// int8_choice.h - which tile an int8 product takes, from its sizes alone (host
// code; the tests read it too).
#pragma once

#include <stdint.h>

namespace mxg {

// Each variant's time is estimated as rounds x (slices x us + extra): tiles over
// the workgroups that run at once, us per slice of 128 k with the chip full
// (seven tenths of it where a variant that fits twice on a CU has it for
// itself), and what a tile costs besides; and as no less than the weights'
// time from memory.  The smallest estimate is taken, the first of equal ones.
// The constants are measured; what the choice is worth, in us (bf16 output,
// operands from memory, calls of one captured graph; dense M x N x K, or tokens
// x choices of experts of N x K; * what is taken, at most 7 % behind the fastest).
// The time of A's and C's bytes is left out.
//                                  16x16  16x32  32x32  32x64   deep 128x128 256x128 256x256
//   16 x 4096 x 4096                 7.1*   8.3    8.5   11.6   18.7    28.1    28.8    43.7
//   16 x 28672 x 8192               49.5   46.3*  53.8   46.1   53.5    59.8    64.7    88.2
//   32 x 28672 x 8192               71.8   59.7   55.4   46.8*  51.9    59.5    63.4    91.1
//   64 x 4096 x 14336               34.9   27.7   22.9*  31.6   58.4    87.3    88.7     142
//   256 x 4096 x 4096               41.8   29.3   27.2   17.4*  22.9    28.9    32.6    49.2
//   1024 x 4096 x 4096               155    105   98.8   54.2   23.9*   29.4    32.2    47.9
//   512 x 14336 x 4096               267    183    171   92.3   46.5    43.0    35.1*   50.9
//   8192 x 14336 x 4096             3824   2528   2588   1301    576     520     454     398*
//   16 x 4 of 64 of 2048 x 4096     92.9   73.2*  93.5   82.3   96.8     104     115     124
//   256 x 4 of 64 of 2048 x 4096     188    134    150    114*   139     148     153     148
//   1024 x 8 of 64 of 2048 x 4096    864    546    544    281    182     168*    164     158
//   2048 x 4 of 16 of 4096 x 2048   1166    651    665    282    139     118*    124     112
struct I8Variant {
  int bm, bn, per_cu;
  double us, extra;
};
// the order is that of the launches in gemm_int8.hip
constexpr I8Variant kI8Variants[] = {
    {16, 16, 2, 0.18, 1.8},   {16, 32, 2, 0.22, 1.8},   {32, 32, 1, 0.19, 2.4},   {32, 64, 2, 0.52, 1.5},
    {128, 128, 1, 0.55, 3.0}, {128, 128, 2, 1.00, 2.0}, {256, 128, 1, 0.87, 3.0}, {256, 256, 1, 1.45, 8.0}};
constexpr int kI8VariantCount = 8;

constexpr int kCus = 256;
constexpr double kBytesPerUs = 5.2e6;

// Time in us; E = 0: a dense product, else M rows over E experts.
inline double i8_estimate(const I8Variant& v, int64_t M, int64_t N, int64_t K, int64_t E) {
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
inline int i8_choice(int64_t M, int64_t N, int64_t K, int64_t E) {
  int best = 0;
  double least = i8_estimate(kI8Variants[0], M, N, K, E);
  for (int v = 1; v < kI8VariantCount; v++) {
    const double t = i8_estimate(kI8Variants[v], M, N, K, E);
    if (t < least) {
      best = v;
      least = t;
    }
  }
  return best;
}

}  // namespace mxg
