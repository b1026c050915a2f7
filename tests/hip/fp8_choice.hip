// The E4M3 products' and weight gradients' choice of a tile, for the tests (host code only).
#include "../../block_scaled_precision_mxgemm_amd/csrc/fp8_choice.h"

extern "C" int fp8_choice(int64_t M, int64_t N, int64_t K, int64_t E) { return mxg::f8_choice(M, N, K, E); }
// splits of the rows, 0 for the large tile
extern "C" int fp8_grad_choice(int64_t M, int64_t N, int64_t K, int64_t E, int terms) {
  const mxg::GradChoice c = mxg::grad_choice(M, N, K, E, terms);
  return c.large ? 0 : c.splits;
}
