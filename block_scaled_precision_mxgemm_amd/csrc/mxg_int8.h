// mxg_int8.h - what the int8 product kernels share: arguments, the MFMA and the
// output step.
//
// Operand layout of v_mfma_i32_16x16x64_i8: lane l holds 16 codes of row
// l % 16; which k of the 64 they are cancels out as long as both operands use
// the same (here lane group l / 16 holds the 16-byte chunk l / 16 of a 64-byte
// step).  Result as for the other 16 x 16 MFMAs: D[4 (l / 16) + i][l % 16],
// rows from the first operand's; with B first a lane holds 4 consecutive
// columns of one row of C.
#pragma once

#include "mxg_experts.h"

namespace mxg {

struct I8Args {
  const int8_t* A;
  const float* SA;
  int64_t rows_a;
  const int8_t* B;          // E x N x K
  const float* SB;          // E x N
  Epi e;                    // e.bias: E x N, or nullptr
  int64_t M;                // rows of C
  int N, K;
  int E;                    // experts; offsets == nullptr: one, all rows
  const int32_t* offsets;   // E + 1
  const int32_t* index;     // M, or nullptr
  int index_div;
  // i / index_div for 0 <= i < 2^31 is i * div_mul >> div_shift (set_division)
  uint32_t div_mul;
  int div_shift;
};

using I8Tile = ExpertTile;

// Scale of that row; rows outside A give NaN.
__device__ __forceinline__ float a_scale(const I8Args& a, int64_t row) {
  return row < 0 ? __builtin_nanf("") : a.SA[row];
}

__device__ __forceinline__ v4i mfma_i8(const v4i& x, const v4i& y, const v4i& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(x, y, c, 0, 0, 0);
}

// Output step of 4 columns n .. n+3 of row m: the sum rounded to fp32 (one
// rounding of at most 2^-24 of it; exact below 2^24), times the row's scale,
// times the column's, then bias, activation and the output type.
__device__ __forceinline__ void store4(const I8Args& a, int expert, int64_t m, int n, const v4i& sum, float s) {
  const int64_t base = (int64_t)expert * a.N;
  const v4f c = load_columns(a.SB + base, n, a.N, 0.0f);
  v4f v;
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = rounded_product(rounded_product((float)sum[i], s), c[i]);
  if (a.e.bias != nullptr) v += load_columns(a.e.bias + base, n, a.N, 0.0f);
  if (a.e.act == kActGelu) {
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = gelu(v[i]);
  }
  store_columns<false>(a.e, a.N, m, n, v);
}

}  // namespace mxg
