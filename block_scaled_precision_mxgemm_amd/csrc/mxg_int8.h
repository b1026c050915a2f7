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

#include "mxg_rows.h"

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

// With 2^(s-1) < d <= 2^s and m = floor(2^(31+s) / d) + 1, m d exceeds 2^(31+s)
// by at most d <= 2^s, so i m / 2^(31+s) exceeds i / d by less than 1 / d for
// i < 2^31, and its floor is that of i / d.
inline void set_division(I8Args& a) {
  int s = 0;
  while (((int64_t)1 << s) < a.index_div) s++;
  a.div_mul = (uint32_t)(((uint64_t)1 << (31 + s)) / (uint32_t)a.index_div + 1);
  a.div_shift = 31 + s;
}

// Tiles of `bm` rows that any offsets can ask for.
inline int64_t i8_tiles_m(const I8Args& a, int bm) {
  const int64_t full = (a.M + bm - 1) / bm;
  // every expert can end in a partial tile; no more tiles than rows
  return a.offsets == nullptr ? full : (full + a.E - 1 < a.M ? full + a.E - 1 : a.M);
}

struct I8Tile {
  int64_t row0;  // first row of C
  int rows;      // rows of this tile
  int expert;
  int tn;        // column tile
};

// Workgroup id -> tile id: workgroups are dispatched round-robin over the 8
// XCDs, so each XCD gets a contiguous range of tile ids; within the range,
// groups of 8 row tiles take the column tiles in turn, so that what runs at
// once on an XCD shares rows of A and of B in its L2.
__device__ __forceinline__ void tile_order(int bid, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int total = tiles_m * tiles_n;
  const int x = bid & 7, rem = total & 7;
  const int id = x * (total >> 3) + min(x, rem) + (bid >> 3);
  const int group = id / (8 * tiles_n);
  const int first = group * 8;
  const int rows = min(tiles_m - first, 8);
  const int in = id - group * 8 * tiles_n;
  tm = first + in % rows;
  tn = in / rows;
}

// Tile `bid` in that order, found by a wave (every lane gets it); false if
// there is none.  By expert, each lane takes a run of experts and the lane
// whose run holds the tile passes it on.  The offsets count as kept inside
// 0 .. M and never falling (each at least the largest before it), so that
// whatever they hold, no row has two experts.
__device__ __forceinline__ bool find_tile(const I8Args& a, int bm, int tiles_n, int64_t bid, int lane, I8Tile& t) {
  const int M = (int)a.M;
  int tm;
  if (a.offsets == nullptr) {
    const int tiles_m = (M + bm - 1) / bm;
    if (bid >= (int64_t)tiles_m * tiles_n) return false;
    tile_order((int)bid, tiles_m, tiles_n, tm, t.tn);
    t.row0 = (int64_t)tm * bm;
    t.rows = min(M - tm * bm, bm);
    t.expert = 0;
    return true;
  }
  const int per = (a.E + 63) / 64;
  const int e0 = lane * per, e1 = min(e0 + per, a.E);
  // first row of the run: the largest offset up to e0
  int top = 0;
  for (int e = e0; e < e1; e++) top = max(top, min(a.offsets[e + 1], M));
  if (lane == 0) top = max(top, min(a.offsets[0], M));
  top = wave_scan<true>(top);
  int first = __shfl_up(top, 1);
  if (lane == 0) first = max(0, min(a.offsets[0], M));
  int mine = 0;
  int lo = first;
  for (int e = e0; e < e1; e++) {
    const int hi = max(lo, min(a.offsets[e + 1], M));
    mine += (hi - lo + bm - 1) / bm;
    lo = hi;
  }
  int before = wave_scan<false>(mine);
  const int total = __builtin_amdgcn_readlane(before, 63);
  if (bid >= (int64_t)total * tiles_n) return false;
  tile_order((int)bid, total, tiles_n, tm, t.tn);
  before -= mine;
  int row0 = 0, rows = 0, expert = 0;
  const bool holds = tm >= before && tm < before + mine;
  if (holds) {
    lo = first;
    for (int e = e0; e < e1; e++) {
      const int hi = max(lo, min(a.offsets[e + 1], M));
      const int n = (hi - lo + bm - 1) / bm;
      if (tm < before + n) {
        row0 = lo + (tm - before) * bm;
        rows = min(hi - row0, bm);
        expert = e;
        break;
      }
      before += n;
      lo = hi;
    }
  }
  const int src = __builtin_ctzll(__ballot(holds));
  t.row0 = __builtin_amdgcn_readlane(row0, src);
  t.rows = __builtin_amdgcn_readlane(rows, src);
  t.expert = __builtin_amdgcn_readlane(expert, src);
  return true;
}

// Row of A that row p of C takes; -1 for an index outside A.
__device__ __forceinline__ int64_t a_row(const I8Args& a, int64_t p) {
  if (a.index == nullptr) return p;
  const int i = a.index[p];
  const int64_t row = i < 0 ? -1 : (int64_t)(((uint64_t)(uint32_t)i * a.div_mul) >> a.div_shift);
  return row < a.rows_a ? row : -1;
}

// Scale of that row; rows outside A give NaN.
__device__ __forceinline__ float a_scale(const I8Args& a, int64_t row) {
  return row < 0 ? __builtin_nanf("") : a.SA[row];
}

__device__ __forceinline__ v4i mfma_i8(const v4i& x, const v4i& y, const v4i& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(x, y, c, 0, 0, 0);
}

// A product that is rounded before a sum takes it up (no fma), so that every
// kernel gives the same bits.
__device__ __forceinline__ float rounded_product(float x, float y) {
#pragma clang fp contract(off)
  return x * y;
}

// Vectors at any element's address: rows of C, of the scales and of the bias
// start there when N is not a multiple of 4 (global memory takes such accesses
// in one instruction).
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));
typedef int v2i_any __attribute__((ext_vector_type(2), aligned(2)));

// Values p[0 .. 3] of a row's columns n .. n+3, `other` past its end.
__device__ __forceinline__ v4f load_columns(const float* p, int n, int N, float other) {
  if (n + 3 < N) return *reinterpret_cast<const v4f_any*>(p + n);
  v4f v;
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = n + i < N ? p[n + i] : other;
  return v;
}

// Store of 4 finished values to C[m][n .. n+3]; past the row's end nothing.
template <bool NT>
__device__ __forceinline__ void store_columns(Epi e, int64_t N, int64_t m, int n, v4f v) {
  if (e.out == kOutF32) {
    float* p = reinterpret_cast<float*>(e.C) + m * N + n;
    if (n + 3 < N) {
      if (NT)
        __builtin_nontemporal_store((v4f_any)v, reinterpret_cast<v4f_any*>(p));
      else
        *reinterpret_cast<v4f_any*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 3; i++)
        if (n + i < N) p[i] = v[i];
    }
    return;
  }
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; i++) h[i] = e.out == kOutBF16 ? bf16_bits(v[i]) : f16_bits(v[i]);
  uint16_t* p = reinterpret_cast<uint16_t*>(e.C) + m * N + n;
  if (n + 3 < N) {
    const v2i_any w = {(int)(h[0] | (h[1] << 16)), (int)(h[2] | (h[3] << 16))};
    if (NT)
      __builtin_nontemporal_store(w, reinterpret_cast<v2i_any*>(p));
    else
      *reinterpret_cast<v2i_any*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 3; i++)
      if (n + i < N) p[i] = (uint16_t)h[i];
  }
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
