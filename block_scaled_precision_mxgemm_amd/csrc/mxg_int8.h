// mxg_int8.h - what the int8 product kernels share: arguments, the expert's
// tile of a workgroup, the MFMA and the output step.
//
// Operand layout of v_mfma_i32_16x16x64_i8: lane l holds 16 codes of row
// l % 16; which k of the 64 they are cancels out as long as both operands use
// the same (here lane group l / 16 holds the 16-byte chunk l / 16 of a 64-byte
// step).  Result as for the other 16 x 16 MFMAs: D[4 (l / 16) + i][l % 16],
// rows from the first operand's; with B first a lane holds 4 consecutive
// columns of one row of C.
#pragma once

#include "mxg_epilogue.h"

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
};

// Tiles of `bm` rows that any offsets can ask for.
inline int64_t i8_tiles_m(const I8Args& a, int bm) {
  const int64_t full = (a.M + bm - 1) / bm;
  // every expert can end in a partial tile; no more tiles than rows
  return a.offsets == nullptr ? full : (full + a.E - 1 < a.M ? full + a.E - 1 : a.M);
}

struct I8Tile {
  int64_t row0;  // first row of C
  int rows;      // rows of this tile (0: no such tile)
  int expert;
};

// The tile `tm` of the experts' tiles of bm rows, by one wave: each lane takes
// a run of experts, and the lane whose run holds the tile writes it.  The
// offsets count as kept inside 0 .. M and never falling (each at least the
// largest before it), so that whatever they hold, no row has two experts.
__device__ __forceinline__ void find_tile(const I8Args& a, int bm, int tm, int lane, I8Tile* out) {
  const int M = (int)a.M;
  if (a.offsets == nullptr) {
    if (lane == 0) {
      const int64_t row0 = (int64_t)tm * bm;
      const int64_t left = a.M - row0;
      *out = I8Tile{row0, left < bm ? (int)left : bm, 0};
    }
    return;
  }
  const int per = (a.E + 63) / 64;
  const int e0 = lane * per, e1 = min(e0 + per, a.E);
  // first row of the run: the largest offset up to e0
  int top = 0;
  for (int e = e0; e < e1; e++) top = max(top, min(a.offsets[e + 1], M));
  if (lane == 0) top = max(top, min(a.offsets[0], M));
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(top, d);
    if (lane >= d) top = max(top, o);
  }
  int first = __shfl_up(top, 1);
  if (lane == 0) first = max(0, min(a.offsets[0], M));
  int mine = 0;
  int lo = first;
  for (int e = e0; e < e1; e++) {
    const int hi = max(lo, min(a.offsets[e + 1], M));
    mine += (hi - lo + bm - 1) / bm;
    lo = hi;
  }
  int before = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(before, d);
    if (lane >= d) before += o;
  }
  const int total = __shfl(before, 63);
  before -= mine;
  if (lane == 0 && tm >= total) *out = I8Tile{0, 0, 0};
  if (tm < before || tm >= before + mine) return;
  lo = first;
  for (int e = e0; e < e1; e++) {
    const int hi = max(lo, min(a.offsets[e + 1], M));
    const int n = (hi - lo + bm - 1) / bm;
    if (tm < before + n) {
      const int row0 = lo + (tm - before) * bm;
      *out = I8Tile{row0, min(hi - row0, bm), e};
      return;
    }
    before += n;
    lo = hi;
  }
}

// Row of A that row p of C takes; -1 for an index outside A.
__device__ __forceinline__ int64_t a_row(const I8Args& a, int64_t p) {
  if (a.index == nullptr) return p;
  const int i = a.index[p];
  const int64_t row = i < 0 ? -1 : i / a.index_div;
  return row < a.rows_a ? row : -1;
}

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
  const bool vec = (a.N & 3) == 0;
  Epi e = a.e;
  if (e.bias != nullptr) e.bias += base;
  const float* sb = a.SB + base;
  v4f c = {0.f, 0.f, 0.f, 0.f};
  if (vec) {
    c = *reinterpret_cast<const v4f*>(sb + n);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (n + i < a.N) c[i] = sb[n + i];
  }
  v4f v;
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = ((float)sum[i] * s) * c[i];
  epi_store4<false>(e, a.N, m, n, v, vec);
}

}  // namespace mxg
