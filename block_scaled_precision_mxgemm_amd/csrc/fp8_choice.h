// fp8_choice.h - which tile an E4M3 product with a scale per block of 128 takes,
// from its sizes alone (host code; the tests read it too).
#pragma once

#include <stdint.h>

namespace mxg {

// Each variant's time is estimated as rounds x (blocks x us + extra): tiles over
// the workgroups that run at once, us per block of 128 k with the chip full
// (seven tenths of it where a variant that fits twice on a CU has it for
// itself), and what a tile costs besides; and as no less than the weights'
// time from memory.  The smallest estimate is taken; of equal ones 16 x 32, which
// where memory bounds both is the faster one beside 16 x 16, then the first.
// The constants are measured; what the choice is worth, in us (bf16 output,
// operands from memory, calls of one captured graph; dense M x N x K, or tokens
// x choices of experts of N x K; * what is taken).
//                                  16x16  16x32  32x32  32x64   deep 128x128 256x128 256x256
//   16 x 4096 x 4096                 7.0*   7.8    8.5   13.0   23.5    27.5    31.7    55.1
//   16 x 28672 x 8192               51.1   49.7*  56.6   49.8   58.5    73.1    65.2     109
//   32 x 28672 x 8192               85.5   68.1   62.5   53.2*  55.9    73.1    64.7     109
//   64 x 4096 x 14336               41.1   32.8   25.4*  38.1   79.3     115    97.8     182
//   256 x 4096 x 4096               43.1   31.8   27.4   18.4*  25.8    29.1    38.1    58.1
//   1024 x 4096 x 4096               159    114    102   60.8   27.1*   31.7    38.1    60.2
//   777 x 4100 x 2064               88.0   65.4   60.7   35.3   19.0*   20.2    24.4    38.5
//   512 x 14336 x 4096               298    215    192    115   66.5    54.2*   54.3    67.7
//   2048 x 4096 x 4096                                    117   49.3    40.2    42.0*   60.9
//   8192 x 14336 x 4096                                  1609    758     601     584     443*
//   16 x 4 of 64 of 2048 x 4096     90.2   73.5*  97.2   81.0   95.8     107     110     128
//   256 x 4 of 64 of 2048 x 4096     195    140    152    115*   138     150     158     152
//   1024 x 8 of 64 of 2048 x 4096                  616    343    280     231     201     167*
//   2048 x 4 of 16 of 4096 x 2048                  685    313    151     123     144     125
//   4096 x 4 of 16 of 4096 x 2048                 1325    600    301     237     236     197*
// and 64x128, in a run of its own with some of the others beside it:
//                                  32x64    deep 128x128 256x128  64x128
//   256 x 4096 x 4096               21.0*   36.2    36.8    55.0    22.8
//   512 x 4096 x 4096               36.9    34.2    36.2    49.5    22.6*
//   1000 x 2000 x 8192              61.0    56.6    68.2    87.3    38.7*
//   1024 x 4096 x 4096              66.5    33.2*   36.9    47.2    33.8
//   777 x 4100 x 2064               35.0    18.6*   19.3    23.1    20.3
//   500 x 2 of 4 of 2048 x 2048     28.3    21.8*   25.1    33.9    21.9
//   1000 x 2 of 4 of 1024 x 4096    39.4    38.2*   41.3    55.9    30.0
// and few rows over experts, where the estimates are at the weights' time:
//                                  16x16  16x32  32x32  32x64  64x128
//   1 x 8 of 32 of 4096 x 4096      37.8   27.2*   38.2   27.8   29.6
//   4 x 4 of 32 of 4096 x 4096      52.7   40.8*   59.2   43.5   41.5
//   2 x 4 of 64 of 2048 x 4096      22.6   17.7*   22.8   18.9   27.2
//   8 x 4 of 64 of 2048 x 4096      52.9   40.7*   59.5   43.3   41.7
//   4 x 8 of 128 of 1024 x 2048     24.1   17.5*   25.5   16.1   17.8
//   2 x 2 of 8 of 14336 x 4096      60.5   48.6*   65.0   49.0   48.0
struct F8Variant {
  int bm, bn, per_cu;
  double us, extra;
};
// the order is that of the launches in gemm_fp8.hip
constexpr F8Variant kF8Variants[] = {
    {16, 16, 2, 0.21, 1.8},   {16, 32, 2, 0.22, 1.8},   {32, 32, 1, 0.19, 2.4},   {32, 64, 2, 0.48, 1.5},
    {128, 128, 1, 0.72, 4.0}, {128, 128, 2, 1.26, 4.5}, {256, 128, 1, 1.17, 4.0}, {256, 256, 1, 1.85, 7.5},
    {64, 128, 2, 0.80, 3.0}};
constexpr int kF8VariantCount = 9;

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

// Index of the variant with the smallest estimate; of equal ones 16 x 32, then the first.
inline int f8_choice(int64_t M, int64_t N, int64_t K, int64_t E) {
  int best = 1;
  double least = f8_estimate(kF8Variants[1], M, N, K, E);
  for (int v = 0; v < kF8VariantCount; v++) {
    const double t = f8_estimate(kF8Variants[v], M, N, K, E);
    if (t < least) {
      best = v;
      least = t;
    }
  }
  return best;
}

// ---- weight gradients ---------------------------------------------------------
//
// Tiles of 256 x 256 (one workgroup a CU; with dY in two or three terms 256 x 128, two a CU)
// or of 128 x 128 (two a CU), the latter with the rows in up to 64 parts whose
// sums are added by a second kernel.  The estimate: rounds x (slices of 64 rows x us
// + extra), with a CU to itself `alone` instead of `us`; and for parts what a
// launch and the partial sums' bytes take.  Measured, in us (fp32 result; * what is
// taken):
//                              bf16: 256   128  in 2  in 8   fp16: large   128  in 2  in 8   fp32: large   128  in 2  in 8
//   2047 x 4100 x 2064             64.2*  76.2  88.4   166           114*   126   123   165           180*   228   201   241
//   8192 x 4096 x 4096              229*   306   342   507           459*   664   649   743           719*  1059  1077  1172
//   16384 x 1024 x 1024             409    224   118  50.8*          705    545   278   101*         1075    810   411   147*
//   4096 x 2048 x 2048              108   59.3*  52.5  79.4          181    140   103*  113           274    207   148*  169
//   512 x 4096 x 4096              25.9*  28.0  70.3   214          40.4*  48.0  82.0   203          53.8*  74.2   111   229
//   4096 x 4 of 16 of 4096 x 2048   326*   439                       570*   688                       830*  1159
//   4096 x 4 of 32 of 2048 x 1024   122*   146                       168*   198                       236*   320
//   300 x 2 of 8 of 1024 x 1024    16.6   12.9*                     15.2   12.7*                     16.9   14.7*
//   (rows x columns of dY x columns of the codes; tokens x choices of experts of N x K)
//   in more parts, 1 / 4 / 16 / 64 / 256: bf16 16384 x 16 x 64 220 / 61 / 22.5 / 12.2* / 13.1, 16384 x 100 x 512
//   223 / 62 / 23.6 / 15.9* / 31; fp32 the same two 804 / 207 / 59 / 21.1* / 15.1 and 813 / 209 / 60 / 25.7* / 31
constexpr int kGradCus = 256;

struct GradChoice {
  bool large;
  int splits;  // of the rows; > 1: partial sums in the workspace
};

inline GradChoice grad_choice(int64_t M, int64_t N, int64_t K, int64_t E, int terms) {
  auto estimate = [&](bool large, int splits) {
    const int bn = large && terms == 1 ? 256 : 128, bk = large ? 256 : 128;
    const int per_cu = large && terms == 1 ? 1 : 2;
    const double more = terms == 3 ? 1.5 : 1.0;
    const double us = more * (large ? (terms == 1 ? 1.75 : 3.6) : (terms == 1 ? 1.3 : 2.8));
    const double alone = more * (large ? (terms == 1 ? 1.75 : 2.8) : (terms == 1 ? 0.91 : 2.1));
    const double extra = large ? 10.0 : 5.0;
    const double tiles = (double)((N + bn - 1) / bn) * (double)((K + bk - 1) / bk) * (double)E * splits;
    const double full = tiles / (kGradCus * per_cu);
    const double rounds = full > 4.0 ? full + 0.5 : __builtin_ceil(full);
    const double slices = __builtin_ceil((double)M / E / 64.0 / splits);
    const double t = rounds * (slices * (tiles <= kGradCus ? alone : us) + extra);
    return splits == 1 ? t : t + 4.0 + 8.0 * splits * (double)E * N * K / 5.0e6;
  };
  GradChoice best = {true, 1};
  double least = estimate(true, 1);
  for (int splits = 1; splits <= 64; splits *= 2) {
    const double t = estimate(false, splits);
    if (t < least) {
      least = t;
      best = {false, splits};
    }
  }
  return best;
}

}  // namespace mxg
