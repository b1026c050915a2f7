// fp8_weight_grad.hip - the weights' gradient of a product whose activations
// were kept as E4M3 codes with a scale per row and 128 columns:
//   dW[n][k] = sum_m dY[m][n] x[m][k],   x[m][k] = s[m][k / 128] q[m][k],
// dense and by expert (rows offsets[e] .. offsets[e+1] of dY, against rows
// index[p] / index_div of the codes, give dW of expert e).
//
// Products of bf16 values on the bf16 MFMA, summed in fp32.  x is rounded to
// bf16: exact where s is a power of two (a code has 4 significant bits).  dY in
// fp16 is taken as the sum of two bf16 values (TERMS = 2), its nearest one and that of
// the rest (11 bits are 8 and 3), in fp32 as that of three (24 bits).
//
// ANY: scales of any kind, in fp32.  A tile of 128 columns of codes has one scale a row, so
// that it goes with dY instead: fl32(dY s) as three bf16 values, against the codes as they
// are: the MFMAs of dY in fp32 on tiles of 128 x 128, whatever dY's type.  In us, by powers
// of two / others rounded / others in fp32 (dY in bf16; fp16; fp32):
//   8192 x 4096 x 4096             227 / 250 / 1209   455 / 552 / 1188   719 / 802 / 1170
//   2047 x 4100 x 2064            67.2 / 70.9 / 266   118 / 140 / 258    183 / 203 / 269
//   512 x 4096 x 4096            29.7 / 31.1 / 87.3  43.4 / 46.4 / 84.7  57.7 / 63.3 / 87.2
//   4096 x 4 of 16 of 4096 x 2048  322 / 347 / 1333                      828 / 897 / 1347
// (of normal data the rounding is 2^-9.2 of the result, root mean square).
//
// Both operands are contracted over their rows, so that a lane's 8 elements of
// an MFMA operand are a column of LDS: ds_read_b64_tr_b16 reads 4 rows of 16
// columns and hands each lane a column.  Which of the 32 rows of a step an
// element is cancels out, as both operands use the same: rows 4 g .. 4 g + 3
// and 16 + 4 g .. 16 + 4 g + 3 for lanes 16 g .. 16 g + 15.  A row's 32-byte pieces
// (16 columns) are permuted by row % 8, so that the rows that are read at once lie in
// different banks.
//
// 8192 x 4096 x 4096 takes 229 - 243 us (1130 - 1200 TFLOP/s; a large library product of
// bf16 1420).  A loop of the MFMAs and their operands' LDS reads takes 170 of them, the
// barriers 9, the loads 24, the conversion and the writes to LDS 38: the codes come as
// bytes of rows and have to be bf16 in LDS before a lane can read a column, which
// direct global -> LDS copies cannot do.
#include <type_traits>

#include "fp8_choice.h"
#include "mxg_experts.h"
#include "mxg_internal.h"

namespace mxg {
namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) { return bf16_bits(a) | (bf16_bits(b) << 16); }

// bf16 bits of f, and what they leave of it (exactly).  A finite value beyond bf16's range is
// cut off instead of rounded; infinities and NaNs leave nothing.
__device__ __forceinline__ uint32_t split_bf16(float& f) {
  uint32_t h = bf16_bits(f);
  if ((h & 0x7fffu) == 0x7f80u) h = __float_as_uint(f) >> 16;
  const float rest = f - __uint_as_float(h << 16);
  f = rest == rest ? rest : 0.0f;
  return h;
}

// A thread's number in a form that the compiler cannot see through: what is
// derived from it is formed where it is used, and not held in registers
// across the loops.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ void barrier_lds() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Accumulator tied in AGPRs, in program order.
__device__ __forceinline__ void mfma_bf16_acc(v4f& c, const v8s& x, const v8s& y) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(x), "v"(y));
}

// BK x BN of dW by WK x WN waves, each with FK x FN fragments, in slices of MS rows.
template <int BK_, int BN_, int WK_, int WN_, int TERMS_, int MS_>
struct GradCfg {
  static constexpr int MS = MS_;
  static constexpr int BK = BK_, BN = BN_, WK = WK_, WN = WN_, TERMS = TERMS_;
  static constexpr int NT = WK * WN * 64;
  static constexpr int FK = BK / WK / 16, FN = BN / WN / 16;
  static constexpr int PX = BK * 2, PY = BN * 2;  // bytes of a row in LDS
  static constexpr int OFF_Y = MS * PX, SZY = MS * PY, STAGE = OFF_Y + TERMS * SZY;
  static constexpr int LDS = 2 * STAGE;
  static constexpr int PER_CU = LDS > 80 * 1024 ? 1 : 2;
  // pieces of a thread: 16 codes, 8 elements of dY
  static constexpr int CX = MS * BK / 16 / NT, CY = MS * BN / 8 / NT;
  static_assert(LDS <= 160 * 1024, "fits the 160 KiB LDS of a gfx950 CU");
  static_assert(CX * NT * 16 == MS * BK && CY * NT * 8 == MS * BN && FN >= 2, "pieces split evenly");
};

template <int IN, class T, bool GATHER, bool ANY>
struct Grad {
  static constexpr int FK = T::FK, FN = T::FN, TERMS = T::TERMS, COLS = FN * TERMS;
  static_assert(!ANY || (T::BK == 128 && TERMS == 3), "a scale a row, products of it in fp32");
  static constexpr int ROWS = T::CX + (ANY ? T::CY : 0);  // rows of A that a thread looks up for a slice
  static constexpr int kMS = T::MS;
  static constexpr int VY = IN == kOutF32 ? 2 : 1;  // registers of 16 bytes of a piece of dY

  // A slice on its way from memory to LDS.
  struct Held {
    v4i x[T::CX];
    float s[T::CX];
    int bad;  // bit u: the row of x[u] is outside A
    v4i y[T::CY][VY];
    float sy[T::CY];  // ANY: the scales of these rows
  };
  struct Tile {
    int e, k0, n0;
    int m0, m1;  // rows
    int64_t out; // partial sums: which of the splits
  };

  // What a thread keeps of its places in a tile's slices, so that a slice needs no
  // index arithmetic: offsets of its first piece from a slice's first row (those of
  // the others are a whole number of rows behind) and its places in LDS.
  struct Place {
    uint32_t x, s, y;  // elements of A, SA, dY
    int to_x, to_y;    // bytes
  };
  static constexpr int ROWS_X = T::NT * 16 / T::BK, ROWS_Y = T::NT * 8 / T::BN;  // rows between pieces
  static_assert(ROWS_X % 8 == 0 && ROWS_Y % 8 == 0, "pieces of a thread have one permutation");
  static __device__ __forceinline__ Place place(const F8GradArgs& a, const Tile& t) {
    Place w;
    const int tid = opaque(threadIdx.x);
    const int rx = tid / (T::BK / 16), f = tid % (T::BK / 16);
    const int ry = tid / (T::BN / 8), q = tid % (T::BN / 8);
    // (nothing is stored of the columns past K)
    const int k = min(t.k0 + f * 16, a.K - 16);
    w.x = (GATHER ? 0u : (uint32_t)rx * (uint32_t)a.K) + (uint32_t)k;
    w.s = (GATHER ? 0u : (uint32_t)rx * (uint32_t)a.KB) + (uint32_t)(k >> 7);
    w.y = (uint32_t)ry * (uint32_t)a.N + (uint32_t)(t.n0 + q * 8);
    w.to_x = rx * T::PX + ((f ^ (rx & 7)) << 5);
    w.to_y = T::OFF_Y + ry * T::PY + (((q >> 1) ^ (ry & 7)) << 5) + (q & 1) * 16;
    return w;
  }

  static __device__ __forceinline__ void load_index(const F8GradArgs& a, const Tile& t, int m, int (&at)[ROWS]) {
    if constexpr (GATHER) {
#pragma unroll
      for (int u = 0; u < T::CX; u++)
        at[u] = a.index[min(m + (int)threadIdx.x / (T::BK / 16) + u * ROWS_X, t.m1 - 1)];
      if constexpr (ANY) {
#pragma unroll
        for (int u = 0; u < T::CY; u++)
          at[T::CX + u] = a.index[min(m + (int)threadIdx.x / (T::BN / 8) + u * ROWS_Y, t.m1 - 1)];
      }
    }
  }
  // ANY: the scales of dY's rows in the tile's block of columns (rows past m1 take the last one's)
  static __device__ __forceinline__ void load_scales(const F8GradArgs& a, const Tile& t, int m, const int (&at)[ROWS],
                                                     Held& h) {
#pragma unroll
    for (int u = 0; u < T::CY; u++) {
      int64_t row = min(m + opaque(threadIdx.x) / (T::BN / 8) + u * ROWS_Y, t.m1 - 1);
      if constexpr (GATHER) row = row_of_index(a, at[T::CX + u]);
      const float s = a.SA[max(row, (int64_t)0) * a.KB + (t.k0 >> 7)];
      h.sy[u] = row < 0 ? __builtin_nanf("") : s;
    }
  }

  // The pieces of rows m .. m + 63 (m < m1).  Offsets from the slice's first element
  // fit 32 bits (64 rows of 2^20).  FULL: all rows exist and no piece ends behind
  // dY (columns past N hold what follows in memory: nothing of theirs is stored).
  // Else rows past m1 are fetched as the last one, and dY element by element.
  template <bool FULL>
  static __device__ __forceinline__ void load_slice(const F8GradArgs& a, const Tile& t, int m, const Place& w,
                                                    const int (&at)[ROWS], Held& h) {
    using E = typename RowElem<IN>::type;
    const int most = t.m1 - 1 - m;
    h.bad = 0;
#pragma unroll
    for (int u = 0; u < T::CX; u++) {
      if constexpr (GATHER) {
        int64_t row = row_of_index(a, at[u]);
        if (row < 0) h.bad |= 1 << u;
        row = max(row, (int64_t)0);
        h.x[u] = *reinterpret_cast<const v4i*>(a.A + row * a.K + w.x);
        if constexpr (!ANY) h.s[u] = a.SA[row * a.KB + w.s];
      } else {
        uint32_t x = w.x, s = w.s;
        const uint8_t* from_x = a.A + (int64_t)m * a.K;
        const float* from_s = a.SA + (int64_t)m * a.KB;
        if constexpr (FULL) {
          from_x += u * ((int64_t)ROWS_X * a.K);
          from_s += u * ((int64_t)ROWS_X * a.KB);
        } else {
          const int rx = opaque(threadIdx.x) / (T::BK / 16);
          const uint32_t back = (uint32_t)(rx + u * ROWS_X - min(rx + u * ROWS_X, most));
          x += (uint32_t)(u * ROWS_X) * (uint32_t)a.K - back * (uint32_t)a.K;
          s += (uint32_t)(u * ROWS_X) * (uint32_t)a.KB - back * (uint32_t)a.KB;
        }
        h.x[u] = *reinterpret_cast<const v4i*>(from_x + x);
        if constexpr (!ANY) h.s[u] = from_s[s];
      }
    }
    if constexpr (ANY) load_scales(a, t, m, at, h);
    if constexpr (FULL) {
#pragma unroll
      for (int u = 0; u < T::CY; u++) {
        const E* base = (const E*)a.dY + (int64_t)m * a.N + u * ((int64_t)ROWS_Y * a.N);
#pragma unroll
        for (int v = 0; v < VY; v++) h.y[u][v] = *reinterpret_cast<const v4i_any*>(base + w.y + v * RowElem<IN>::VEC);
      }
    } else {
      const E* base = (const E*)a.dY + (int64_t)m * a.N;
      const int64_t left = (a.M - m) * a.N;  // elements from there to the end of dY
      constexpr int PER = 4 / sizeof(E);
#pragma unroll
      for (int u = 0; u < T::CY; u++) {
        const int tid = opaque(threadIdx.x), ry = tid / (T::BN / 8) + u * ROWS_Y;
        const int64_t i = (int64_t)min(ry, most) * a.N + t.n0 + tid % (T::BN / 8) * 8;
#pragma unroll
        for (int d = 0; d < 4 * VY; d++) {
          uint32_t x = 0;
#pragma unroll
          for (int j = 0; j < PER; j++) {
            E one = 0;
            if (i + d * PER + j < left) one = base[i + d * PER + j];
            if constexpr (PER == 1)
              x = __float_as_uint(one);
            else
              x |= (uint32_t)one << (16 * j);
          }
          asm volatile("" : "+v"(x)::"memory");  // one at a time: no registers for all
          h.y[u][d >> 2][d & 3] = (int)x;
        }
      }
    }
  }
  static __device__ __forceinline__ void load(const F8GradArgs& a, const Tile& t, int m, const Place& w,
                                              const int (&at)[ROWS], Held& h) {
    // a row more than the slice's: the last pieces of a row end up to BN - 1 columns behind it
    if (m + kMS <= t.m1 && ((a.M - m - (kMS - 1)) * a.N - t.n0 >= T::BN))
      load_slice<true>(a, t, m, w, at, h);
    else
      load_slice<false>(a, t, m, w, at, h);
  }

  // The pieces into their stage; `rows`: those that count, the others become zeros
  // (FULL: all count).
  template <bool FULL>
  static __device__ __forceinline__ void put_rows(const Held& h, const Place& w, uint8_t* stage, int rows) {
    // Scales that are powers of two (within 2^+-100) are applied by the conversion
    // itself, exactly: 8 instructions where the products and their rounding take 32.
    bool simple = true;
    float s[T::CX];
#pragma unroll
    for (int u = 0; u < T::CX; u++) {
      // (ANY: a row outside A is NaN by dY's scale)
      s[u] = ANY ? 1.0f : GATHER && (h.bad >> u & 1) ? __builtin_nanf("") : h.s[u];
      const uint32_t bits = __float_as_uint(s[u]);
      simple = simple && (bits & 0x7fffffu) == 0u && bits - 0x0d800000u <= 0x64000000u;
    }
    v4i out[T::CX][2];
    if (__all(simple)) {
#pragma unroll
      for (int u = 0; u < T::CX; u++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          out[u][j >> 1][2 * (j & 1)] =
              __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)h.x[u][j], s[u], false));
          out[u][j >> 1][2 * (j & 1) + 1] =
              __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)h.x[u][j], s[u], true));
        }
    } else {
#pragma unroll
      for (int u = 0; u < T::CX; u++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(h.x[u][j], false);
          const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(h.x[u][j], true);
          out[u][j >> 1][2 * (j & 1)] = (int)pack_bf16(lo[0] * s[u], lo[1] * s[u]);
          out[u][j >> 1][2 * (j & 1) + 1] = (int)pack_bf16(hi[0] * s[u], hi[1] * s[u]);
        }
    }
    v4i y[T::CY][TERMS];
#pragma unroll
    for (int u = 0; u < T::CY; u++) {
      if constexpr (TERMS == 1) {
        y[u][0] = h.y[u][0];  // bf16 as it is
      } else {
        float f[8];
        if constexpr (IN == kOutF32) {
#pragma unroll
          for (int j = 0; j < 8; j++) f[j] = __int_as_float(h.y[u][j >> 2][j & 3]);
        } else {
          unpack16<IN>(h.y[u][0], f);
        }
        if constexpr (ANY) {
#pragma unroll
          for (int j = 0; j < 8; j++) f[j] *= h.sy[u];
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
#pragma unroll
          for (int v = 0; v < TERMS - 1; v++) y[u][v][j] = (int)(split_bf16(f[2 * j]) | (split_bf16(f[2 * j + 1]) << 16));
          y[u][TERMS - 1][j] = (int)pack_bf16(f[2 * j], f[2 * j + 1]);
        }
      }
    }
    if constexpr (!FULL) {
      const int tid = opaque(threadIdx.x);
#pragma unroll
      for (int u = 0; u < T::CX; u++)
        if (tid / (T::BK / 16) + u * ROWS_X >= rows) out[u][0] = out[u][1] = v4i{0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < T::CY; u++)
        if (tid / (T::BN / 8) + u * ROWS_Y >= rows) {
#pragma unroll
          for (int v = 0; v < TERMS; v++) y[u][v] = v4i{0, 0, 0, 0};
        }
    }
#pragma unroll
    for (int u = 0; u < T::CX; u++) {
      v4i* to = reinterpret_cast<v4i*>(stage + w.to_x + u * ROWS_X * T::PX);
      to[0] = out[u][0];
      to[1] = out[u][1];
    }
#pragma unroll
    for (int u = 0; u < T::CY; u++)
#pragma unroll
      for (int v = 0; v < TERMS; v++)
        *reinterpret_cast<v4i*>(stage + w.to_y + u * ROWS_Y * T::PY + v * T::SZY) = y[u][v];
  }

  static __device__ __forceinline__ void put(const Held& h, const Place& w, uint8_t* stage, int rows) {
    if (rows >= kMS)
      put_rows<true>(h, w, stage, rows);
    else
      put_rows<false>(h, w, stage, rows);
  }

  static __device__ __forceinline__ v4s read_tr(const uint8_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(p));
  }
  // Operand of a step: 16 columns of 32 rows from p, the lane's place in them.
  static __device__ __forceinline__ v8s operand(const uint8_t* p, int pitch) {
    const v4s lo = read_tr(p), hi = read_tr(p + 16 * pitch);
    return v8s{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  }

  static __device__ __forceinline__ void run(const F8GradArgs& a, int tiles_k, int tiles_n, int splits) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wk = wave / T::WN, wn = wave % T::WN;
    const int g = lane >> 4, i16 = lane & 15;
    const int per = tiles_k * tiles_n, total = per * a.E * splits;

    // Tile number b: workgroups are dispatched round-robin over the 8 XCDs.  Each
    // XCD gets an eighth of every expert's tiles (their numbers of rows differ),
    // or a contiguous range where they do not split evenly; in an expert, groups of
    // 4 tiles of columns of dY take the tiles of codes in turn.
    auto find = [&](int b, Tile& t) {
      const int x = b & 7, rem = total & 7;
      int which, in;
      if (per % 8 == 0) {
        which = (b >> 3) / (per >> 3);
        in = (b >> 3) - which * (per >> 3) + x * (per >> 3);
      } else {
        const int id = x * (total >> 3) + min(x, rem) + (b >> 3);
        which = id / per;
        in = id - which * per;
      }
      const int e = which / splits, z = which - e * splits;
      const int group = in / (4 * tiles_k), first = group * 4, rows = min(tiles_n - first, 4);
      const int rest = in - group * 4 * tiles_k;
      int lo = 0, hi = (int)a.M;
      if (a.offsets != nullptr) {
        // the offsets count as kept inside 0 .. M and never falling
        int top = 0;
        for (int i = lane; i <= e; i += 64) top = max(top, min(a.offsets[i], (int)a.M));
        top = __builtin_amdgcn_readlane(wave_scan<true>(top), 63);
        lo = top;
        hi = max(lo, min(a.offsets[e + 1], (int)a.M));
      }
      // the expert's rows in `splits` parts of whole slices
      const int part = ((hi - lo + kMS - 1) / kMS + splits - 1) / splits * kMS;
      t.e = e;
      t.n0 = (first + rest % rows) * T::BN;
      t.k0 = rest / rows * T::BK;
      t.m0 = __builtin_amdgcn_readfirstlane(min(lo + z * part, hi));
      t.m1 = __builtin_amdgcn_readfirstlane(min(lo + (z + 1) * part, hi));
      t.out = (int64_t)z * a.E + e;
    };

    Tile t;
    find(blockIdx.x, t);
    Held h[2];
    int at[ROWS];
    Place w;
    // the lane's place in a fragment's rows; column f is at that ^ (f << 5)
    const int row = 4 * g + (i16 >> 2);
    const int px = row * T::PX + ((row & 7) << 5) + (i16 & 3) * 8;
    const int py = row * T::PY + ((row & 7) << 5) + (i16 & 3) * 8;
    auto start = [&](const Tile& t) {
      w = place(a, t);
      // slices 0 and 1, and the rows of slice 2
#pragma unroll
      for (int i = 0; i < 2; i++) {
        if (t.m0 + i * kMS < t.m1) {
          load_index(a, t, t.m0 + i * kMS, at);
          load(a, t, t.m0 + i * kMS, w, at, h[i]);
        }
      }
      if (t.m0 + 2 * kMS < t.m1) load_index(a, t, t.m0 + 2 * kMS, at);
    };
    start(t);

    const int S = (t.m1 - t.m0 + kMS - 1) / kMS;
    v4f acc[FK][FN];
#pragma unroll
    for (int i = 0; i < FK; i++)
#pragma unroll
      for (int j = 0; j < FN; j++) {
        acc[i][j] = v4f{0, 0, 0, 0};
        asm volatile("" : "+a"(acc[i][j]));
      }
    asm volatile("s_nop 7" ::: "memory");
    // slice s into stage s % 2, and slice s + 2 on its way
    auto stage_in = [&](int s, Held& held) {
      put(held, w, smem + (s & 1) * T::STAGE, t.m1 - t.m0 - s * kMS);
      if (s + 2 < S) {
        const int m = t.m0 + (s + 2) * kMS;
        load(a, t, m, w, at, held);
        if (s + 3 < S) load_index(a, t, m + kMS, at);
      }
    };
    // MFMAs of 32 rows of slice s
    auto multiply = [&](int s, int step) {
      const uint8_t* stage = smem + (s & 1) * T::STAGE;
      auto column = [&](int c) {
        return operand(stage + T::OFF_Y + (c / FN) * T::SZY + step * 32 * T::PY + (py ^ ((wn * FN + c % FN) << 5)), T::PY);
      };
      v8s fx[FK], fy[2];
#pragma unroll
      for (int i = 0; i < FK; i++) fx[i] = operand(stage + step * 32 * T::PX + (px ^ ((wk * FK + i) << 5)), T::PX);
      fy[0] = column(0);
      fy[1] = column(1);
#pragma unroll
      for (int c = 0; c < COLS; c++) {
#pragma unroll
        for (int i = 0; i < FK; i++) mfma_bf16_acc(acc[i][c % FN], fx[i], fy[c & 1]);
        __builtin_amdgcn_sched_barrier(0);
        if (c + 2 < COLS) fy[c & 1] = column(c + 2);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // Slice s, and slice s + 1 into the other stage.  Where two waves of a workgroup
    // share a SIMD they do the latter at different times, so that one converts
    // while the other, which goes first then, multiplies.
    auto slice = [&](int s, Held& held) {
      const bool more = s + 1 < S;
      constexpr int STEPS = kMS / 32;
      const bool late = T::NT > 256 && STEPS == 2 && wave >= T::NT / 128;
      if (more && !late) stage_in(s + 1, held);
      asm volatile("s_setprio 1");
      multiply(s, 0);
      asm volatile("s_setprio 0");
      if (more && late) stage_in(s + 1, held);
      if constexpr (STEPS == 2) {
        asm volatile("s_setprio 1");
        multiply(s, 1);
        asm volatile("s_setprio 0");
      }
      barrier_lds();
    };
    if (S > 0) {
      stage_in(0, h[0]);
      barrier_lds();
      for (int s = 0; s < S; s += 2) {
        slice(s, h[1]);
        if (s + 1 < S) slice(s + 1, h[0]);
      }
    }
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    if (splits > 1 || a.out_type == kOutF32)
      store32(splits > 1 ? a.workspace : a.dW, a, t, acc, smem + wave * 4096, wk, wn);
    else if (a.out_type == kOutBF16)
      store16<kOutBF16>(a, t, acc, smem, wk, wn);
    else
      store16<kOutF16>(a, t, acc, smem, wk, wn);
  }

  // Output: a lane holds columns 4 g .. 4 g + 3 of row lane % 16 of each fragment.
  // fp32: 16 rows of a wave's 64 columns at a time go through 4 KiB of LDS and come back
  // with 16 lanes on a row, so that the stores fill lines.
  static __device__ __forceinline__ void store32(void* out, const F8GradArgs& a, const Tile& t, v4f (&acc)[FK][FN],
                                                 uint8_t* cst, int wk, int wn) {
    static_assert(FK == 4 && T::NT * 64 <= T::LDS, "64 columns a wave; staging of all waves");
    const int lane = opaque(threadIdx.x & 63), g = lane >> 4, i16 = lane & 15;
    const int k = t.k0 + wk * 64 + i16 * 4;
    float* const base = (float*)out + t.out * a.N * a.K + k;
#pragma unroll
    for (int j = 0; j < FN; j++) {
#pragma unroll
      for (int i = 0; i < FK; i++) {
        asm volatile("" : "+a"(acc[i][j]));
        *reinterpret_cast<v4f*>(cst + i16 * 256 + (((i * 4 + g) ^ i16) << 4)) = acc[i][j];
      }
      wave_sync();
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int row = q * 4 + g, n = t.n0 + (wn * FN + j) * 16 + row;
        const v4f v = *reinterpret_cast<const v4f*>(cst + row * 256 + ((i16 ^ row) << 4));
        if (n < a.N && k < a.K) __builtin_nontemporal_store(v, reinterpret_cast<v4f*>(base + (int64_t)n * a.K));
      }
      wave_sync();
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // 16 bits: the whole tile goes through LDS and comes back in rows of 256 or 512
  // bytes (a wave's 128 bytes alone are slower than fp32's 256).
  // 4096 tokens x 4 over 16 experts of 4096 x 2048, in us: from the fragments 382 fp32, 440
  // bf16; a wave's columns 349, 376; the tile 359, 338; without any stores 311.
  template <int OUT>
  static __device__ __forceinline__ void store16(const F8GradArgs& a, const Tile& t, v4f (&acc)[FK][FN], uint8_t* smem,
                                                 int wk, int wn) {
    constexpr int PITCH = T::BK * 2, CH = PITCH / 16;  // chunks of a row
    static_assert(T::BN * PITCH <= T::LDS && CH % 16 == 0 && T::NT % CH == 0, "staging of the tile");
    const int tid = opaque(threadIdx.x), g = (tid & 63) >> 4, i16 = tid & 15;
#pragma unroll
    for (int j = 0; j < FN; j++) {
      uint8_t* const to = smem + ((wn * FN + j) * 16 + i16) * PITCH + (g & 1) * 8;
#pragma unroll
      for (int i = 0; i < FK; i++) {
        asm volatile("" : "+a"(acc[i][j]));
        uint32_t b[4];
#pragma unroll
        for (int x = 0; x < 4; x++) b[x] = OUT == kOutBF16 ? bf16_bits(acc[i][j][x]) : f16_bits(acc[i][j][x]);
        *reinterpret_cast<v2i*>(to + ((((wk * FK + i) * 2 + (g >> 1)) ^ i16) << 4)) =
            v2i{(int)(b[0] | (b[1] << 16)), (int)(b[2] | (b[3] << 16))};
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    barrier_lds();
    const int chunk = tid % CH, k = t.k0 + chunk * 8;
    uint16_t* const base = (uint16_t*)a.dW + t.out * a.N * a.K + k;
#pragma unroll 4
    for (int r = tid / CH; r < T::BN; r += T::NT / CH) {
      const v4i v = *reinterpret_cast<const v4i*>(smem + r * PITCH + ((chunk ^ (r & 15)) << 4));
      const int n = t.n0 + r;
      if (n < a.N && k < a.K) __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(base + (int64_t)n * a.K));
    }
  }
};

template <int IN, class T, bool GATHER>
__global__ __launch_bounds__(T::NT) __attribute__((amdgpu_waves_per_eu(2))) void fp8_weight_grad_kernel(
    F8GradArgs a, int tiles_k, int tiles_n, int splits) {
  Grad<IN, T, GATHER, false>::run(a, tiles_k, tiles_n, splits);
}
template <int IN, class T, bool GATHER>
__global__ __launch_bounds__(T::NT) __attribute__((amdgpu_waves_per_eu(2))) void fp8_weight_grad_any_kernel(
    F8GradArgs a, int tiles_k, int tiles_n, int splits) {
  Grad<IN, T, GATHER, true>::run(a, tiles_k, tiles_n, splits);
}

// dW = sum over the splits: each of 4 waves adds every fourth one for 256 elements, 8
// of them on their way at once (2048 x 16 x 64 in 32 parts: 8.6 us with the products, 19.6
// with one after the other; 16384 x 16 x 64 in 64 parts 11.9, 34.3).
__global__ __launch_bounds__(256) void fp8_weight_grad_sum_kernel(const float* part, int splits, int64_t n, void* dW,
                                                                  int type) {
  __shared__ __attribute__((aligned(16))) v4f sums[3][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t i = ((int64_t)blockIdx.x * 64 + lane) * 4;
  v4f s = {0, 0, 0, 0};
  if (i < n) {
#pragma unroll 8
    for (int z = wave; z < splits; z += 4) s += *reinterpret_cast<const v4f*>(part + z * n + i);
  }
  if (wave > 0) sums[wave - 1][lane] = s;
  __syncthreads();
  if (wave > 0 || i >= n) return;
#pragma unroll
  for (int w = 0; w < 3; w++) s += sums[w][lane];
  store_columns<false>(Epi{(uint8_t*)dW + i * epi_elem_bytes(type), nullptr, type, kActNone}, 4, 0, 0, s);
}

template <int IN, class T, bool ANY>
hipError_t launch_tiles(const F8GradArgs& a, int splits, hipStream_t stream) {
  const int tiles_n = (a.N + T::BN - 1) / T::BN, tiles_k = (a.K + T::BK - 1) / T::BK;
  const int64_t tiles = (int64_t)tiles_n * tiles_k * a.E * splits;
  if (tiles * T::NT > 0xffffffffll) return hipErrorInvalidConfiguration;  // threads of a launch
  const dim3 grid((unsigned)tiles), block(T::NT);
  const bool gather = a.index != nullptr;
  if constexpr (ANY) {
    const auto kernel = gather ? fp8_weight_grad_any_kernel<IN, T, true> : fp8_weight_grad_any_kernel<IN, T, false>;
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, tiles_k, tiles_n, splits);
  } else {
    const auto kernel = gather ? fp8_weight_grad_kernel<IN, T, true> : fp8_weight_grad_kernel<IN, T, false>;
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, tiles_k, tiles_n, splits);
  }
  return hipGetLastError();
}

hipError_t add_parts(const F8GradArgs& a, int splits, hipStream_t stream) {
  if (splits == 1) return hipSuccess;
  const int64_t n = (int64_t)a.E * a.N * a.K;
  hipLaunchKernelGGL(fp8_weight_grad_sum_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream,
                     (const float*)a.workspace, splits, n, a.dW, a.out_type);
  return hipGetLastError();
}

template <int IN>
hipError_t launch_in(const F8GradArgs& a, bool any_scale, hipStream_t stream) {
  if (any_scale) {
    // tiles of 128 x 128, in as many parts as the three terms of fp32 take (a workspace of theirs)
    const GradChoice c = grad_choice(a.M, a.N, a.K, a.E, 3);
    const int splits = c.large ? 1 : c.splits;
    const hipError_t e = launch_tiles<IN, GradCfg<128, 128, 2, 2, 3, 32>, true>(a, splits, stream);
    return e != hipSuccess ? e : add_parts(a, splits, stream);
  }
  constexpr int TERMS = IN == kOutBF16 ? 1 : IN == kOutF16 ? 2 : 3;
  // (two workgroups a CU where dY is more than one term)
  using Large = typename std::conditional<TERMS == 1, GradCfg<256, 256, 4, 2, 1, 64>, GradCfg<256, 128, 4, 1, TERMS, 32>>::type;
  using Small = GradCfg<128, 128, 2, 2, TERMS, TERMS == 1 ? 64 : 32>;
  const GradChoice c = grad_choice(a.M, a.N, a.K, a.E, TERMS);
  if (c.large) return launch_tiles<IN, Large, false>(a, 1, stream);
  const hipError_t e = launch_tiles<IN, Small, false>(a, c.splits, stream);
  return e != hipSuccess ? e : add_parts(a, c.splits, stream);
}

}  // namespace

// The workspace is as large for any type of dY.
int64_t fp8_weight_grad_bytes(int64_t M, int64_t N, int64_t K, int64_t E) {
  int64_t most = 0;
  for (int terms = 1; terms <= 3; terms++) {
    const GradChoice c = grad_choice(M, N, K, E, terms);
    if (c.splits > 1 && c.splits * E * N * K * 4 > most) most = c.splits * E * N * K * 4;
  }
  return most;
}

hipError_t launch_fp8_weight_grad(const F8GradArgs& args, int y_type, bool any_scale, hipStream_t stream) {
  F8GradArgs a = args;
  set_division(a);
  if (y_type == kOutF32) return launch_in<kOutF32>(a, any_scale, stream);
  if (y_type == kOutBF16) return launch_in<kOutBF16>(a, any_scale, stream);
  return launch_in<kOutF16>(a, any_scale, stream);
}

}  // namespace mxg
