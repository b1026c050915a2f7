// The int8 products' choice of a tile, for the tests (host code only).
#include "../../block_scaled_precision_mxgemm_amd/csrc/int8_choice.h"

extern "C" int int8_choice(int64_t M, int64_t N, int64_t K, int64_t E) { return mxg::i8_choice(M, N, K, E); }
extern "C" double int8_estimate(int v, int64_t M, int64_t N, int64_t K, int64_t E) {
  return mxg::i8_estimate(mxg::kI8Variants[v], M, N, K, E);
}
