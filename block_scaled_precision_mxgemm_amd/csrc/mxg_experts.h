// mxg_experts.h - what the products by expert share, whatever their operands:
// the expert's tile of a workgroup, the row of A that a row of C takes, and
// the loads and stores of rows that start at any element.
//
// Args has M (rows of C), rows_a (rows of A), N, E, offsets (E + 1, or nullptr:
// one expert that has all rows), index (M, or nullptr), index_div, div_mul and
// div_shift.
#pragma once

#include "mxg_rows.h"

namespace mxg {

// With 2^(s-1) < d <= 2^s and m = floor(2^(31+s) / d) + 1, m d exceeds 2^(31+s)
// by at most d <= 2^s, so i m / 2^(31+s) exceeds i / d by less than 1 / d for
// i < 2^31, and its floor is that of i / d.
template <class Args>
inline void set_division(Args& a) {
  int s = 0;
  while (((int64_t)1 << s) < a.index_div) s++;
  a.div_mul = (uint32_t)(((uint64_t)1 << (31 + s)) / (uint32_t)a.index_div + 1);
  a.div_shift = 31 + s;
}

// Tiles of `bm` rows that any offsets can ask for.
template <class Args>
inline int64_t expert_tiles_m(const Args& a, int bm) {
  const int64_t full = (a.M + bm - 1) / bm;
  // every expert can end in a partial tile; no more tiles than rows
  return a.offsets == nullptr ? full : (full + a.E - 1 < a.M ? full + a.E - 1 : a.M);
}

struct ExpertTile {
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

// The experts' rows as the lanes of a wave hold them: each lane has a run of
// `per` experts.  The offsets count as kept inside 0 .. M and never falling (each
// at least the largest before it), so that whatever they hold, no row has two
// experts.
struct ExpertScan {
  int first;   // first row of the run
  int last;    // and the row behind the last one
  int before;  // tiles of the experts before the run
  int mine;    // and of the run
  int total;   // of all
};

template <class Args>
__device__ __forceinline__ ExpertScan scan_experts(const Args& a, int bm, int lane) {
  ExpertScan s = {0, 0, 0, 0, 0};
  if (a.offsets == nullptr) return s;
  const int M = (int)a.M;
  const int per = (a.E + 63) / 64;
  const int e0 = lane * per, e1 = min(e0 + per, a.E);
  // first row of the run: the largest offset up to e0
  int top = 0;
  for (int e = e0; e < e1; e++) top = max(top, min(a.offsets[e + 1], M));
  if (lane == 0) top = max(top, min(a.offsets[0], M));
  top = wave_scan<true>(top);
  s.first = __shfl_up(top, 1);
  if (lane == 0) s.first = max(0, min(a.offsets[0], M));
  s.last = s.first;
  for (int e = e0; e < e1; e++) {
    const int hi = max(s.last, min(a.offsets[e + 1], M));
    s.mine += (hi - s.last + bm - 1) / bm;
    s.last = hi;
  }
  s.before = wave_scan<false>(s.mine);
  s.total = __builtin_amdgcn_readlane(s.before, 63);
  s.before -= s.mine;
  return s;
}

// Tile `bid` in the order above (every lane gets it); false if there is none.
// By expert, the lane whose run holds the tile passes it on.
template <class Args>
__device__ __forceinline__ bool pick_tile(const Args& a, const ExpertScan& s, int bm, int tiles_n, int64_t bid, int lane,
                                          ExpertTile& t) {
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
  if (bid >= (int64_t)s.total * tiles_n) return false;
  tile_order((int)bid, s.total, tiles_n, tm, t.tn);
  const int per = (a.E + 63) / 64;
  int row0 = 0, rows = 0, expert = 0;
  const bool holds = tm >= s.before && tm < s.before + s.mine;
  if (holds) {
    int lo = s.first, before = s.before;
    if (per == 1) {
      row0 = lo + (tm - before) * bm;
      rows = min(s.last - row0, bm);
      expert = lane;
    } else {
      const int e0 = lane * per, e1 = min(e0 + per, a.E);
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
  }
  const int src = __builtin_ctzll(__ballot(holds));
  t.row0 = __builtin_amdgcn_readlane(row0, src);
  t.rows = __builtin_amdgcn_readlane(rows, src);
  t.expert = __builtin_amdgcn_readlane(expert, src);
  return true;
}

template <class Args>
__device__ __forceinline__ bool find_tile(const Args& a, int bm, int tiles_n, int64_t bid, int lane, ExpertTile& t) {
  return pick_tile(a, scan_experts(a, bm, lane), bm, tiles_n, bid, lane, t);
}

// Row of A that an index stands for; -1 for one outside A.
template <class Args>
__device__ __forceinline__ int64_t row_of_index(const Args& a, int i) {
  const int64_t row = i < 0 ? -1 : (int64_t)(((uint64_t)(uint32_t)i * a.div_mul) >> a.div_shift);
  return row < a.rows_a ? row : -1;
}
// Row of A that row p of C takes.
template <class Args>
__device__ __forceinline__ int64_t a_row(const Args& a, int64_t p) {
  return a.index == nullptr ? p : row_of_index(a, a.index[p]);
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

}  // namespace mxg
