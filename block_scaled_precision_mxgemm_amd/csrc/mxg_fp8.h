// mxg_fp8.h - what the E4M3 product kernels with a scale per block of 128
// share: arguments, the MFMA of a block and the output step.
//
// A block's partial sum is one v_mfma_f32_16x16x128_f8f6f4 (operand layout in
// mxg_device.h; which k a lane's bytes are cancels out as long as both operands
// use the same).  It is added to the accumulator times the block's scales:
// one fp32 fma for each 128 products.
#pragma once

#include "mxg_experts.h"

namespace mxg {

struct F8Args {
  const uint8_t* A;         // rows_a x K
  const float* SA;          // rows_a x KB
  int64_t rows_a;
  const uint8_t* B;         // E x N x K
  const float* SB;          // E x NB x KB
  Epi e;                    // e.bias: E x N, or nullptr
  int64_t M;                // rows of C
  int N, K;
  int E;                    // experts; offsets == nullptr: one, all rows
  const int32_t* offsets;   // E + 1
  const int32_t* index;     // M, or nullptr
  int index_div;
  uint32_t div_mul;         // as in I8Args
  int div_shift;
  int KB, NB;               // blocks of 128 along K and N
};

// Partial sum of one block, with the wait states that the compiler does not
// know of (operands written by VALU instructions before, the result read by
// them behind).
__device__ __forceinline__ v4f mfma_block(const v8i& x, const v8i& y) {
  v4f p;
  asm volatile("s_nop 1\n\tv_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, 0\n\ts_nop 15\n\ts_nop 2"
               : "=&v"(p)
               : "v"(x), "v"(y));
  return p;
}

__device__ __forceinline__ v8i join(const v4i& lo, const v4i& hi) {
  return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// Output step of 4 columns n .. n+3 of row m: bias, activation, output type.
template <bool NT>
__device__ __forceinline__ void f8_store4(const F8Args& a, int expert, int64_t m, int n, v4f v) {
  if (a.e.bias != nullptr) v += load_columns(a.e.bias + (int64_t)expert * a.N, n, a.N, 0.0f);
  if (a.e.act == kActGelu) {
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = gelu(v[i]);
  }
  store_columns<NT>(a.e, a.N, m, n, v);
}

}  // namespace mxg
