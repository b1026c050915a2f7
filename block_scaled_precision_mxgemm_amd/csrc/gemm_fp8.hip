// gemm_fp8.hip - E4M3 x E4M3 products with one fp32 scale per row of A and
// 128 columns, and per 128 x 128 block of B, dense and by expert:
//   C[i][j] = out(act(sum_b (sA[i][b] sB[j / 128][b]) p_b[i][j] + bias_j)),
//   p_b = sum_{k in block b} a_ik b_jk.
// The scales of a block are multiplied in fp32, p_b (an MFMA's sum) times that
// is added to the fp32 accumulator by an fma, block after block.
//
// By expert, rows and offsets are as in gemm_int8.hip.
#include "fp8_choice.h"
#include "mxg_fp8.h"
#include "mxg_internal.h"

namespace mxg {
namespace {

// ---- gathered rows of an A of 4 GiB and more --------------------------------
//
// The one case that the kernels below, whose gathered rows are 32-bit offsets,
// do not take.  64 x 64 tiles, 4 waves of 32 x 32, a block of 128 k at a time
// through registers.
constexpr int kBM = 64, kBN = 64, kBK = 128;

__global__ __launch_bounds__(256) void fp8_tile_kernel(F8Args a, int tiles_n) {
  __shared__ __attribute__((aligned(16))) uint8_t sa[kBM * kBK], sb[kBN * kBK];
  __shared__ int64_t arow[kBM];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, r = lane & 15;
  ExpertTile t;
  for (int64_t tile = blockIdx.x; find_tile(a, kBM, tiles_n, tile, lane, t); tile += gridDim.x) {
    __syncthreads();  // the rows of the tile before have been looked up by all
    if (tid < kBM) arow[tid] = tid < t.rows ? a_row(a, t.row0 + tid) : -1;
    __syncthreads();
    const uint8_t* B = a.B + (int64_t)t.expert * a.N * a.K;
    const int n0 = t.tn * kBN;
    const float* SB = a.SB + ((int64_t)t.expert * a.NB + n0 / 128) * a.KB;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    const int64_t ar0 = arow[wm + r], ar1 = arow[wm + 16 + r];
    v4f acc[2][2] = {};
    for (int b = 0; b < a.KB; b++) {
      for (int c = tid; c < kBM * 8; c += 256) {
        const int row = c >> 3, ch = c & 7, k = b * kBK + ch * 16;
        const int64_t ar = arow[row];
        v4i va = {0, 0, 0, 0}, vb = {0, 0, 0, 0};
        if (ar >= 0 && k < a.K) va = *reinterpret_cast<const v4i*>(a.A + ar * a.K + k);
        if (n0 + row < a.N && k < a.K) vb = *reinterpret_cast<const v4i*>(B + (int64_t)(n0 + row) * a.K + k);
        const int o = row * kBK + ((ch ^ swz8(row)) << 4);
        *reinterpret_cast<v4i*>(sa + o) = va;
        *reinterpret_cast<v4i*>(sb + o) = vb;
      }
      const float s = SB[b];
      // rows outside A give NaN
      const float s0 = (ar0 >= 0 ? a.SA[ar0 * a.KB + b] : __builtin_nanf("")) * s;
      const float s1 = (ar1 >= 0 ? a.SA[ar1 * a.KB + b] : __builtin_nanf("")) * s;
      __syncthreads();
      v8i fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int ra = wm + 16 * i + r, rb = wn + 16 * i + r;
        fa[i] = join(*reinterpret_cast<const v4i*>(sa + ra * kBK + ((g ^ swz8(ra)) << 4)),
                     *reinterpret_cast<const v4i*>(sa + ra * kBK + (((4 + g) ^ swz8(ra)) << 4)));
        fb[i] = join(*reinterpret_cast<const v4i*>(sb + rb * kBK + ((g ^ swz8(rb)) << 4)),
                     *reinterpret_cast<const v4i*>(sb + rb * kBK + (((4 + g) ^ swz8(rb)) << 4)));
      }
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const v4f p = mfma_block(fb[j], fa[i]);
#pragma unroll
          for (int x = 0; x < 4; x++) acc[i][j][x] = fmaf(p[x], i == 0 ? s0 : s1, acc[i][j][x]);
        }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int row = wm + 16 * i + r;
      if (row >= t.rows) continue;
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const int n = n0 + wn + 16 * j + 4 * g;
        if (n < a.N) f8_store4<false>(a, t.expert, t.row0 + row, n, acc[i][j]);
      }
    }
  }
}

// 16 bytes at any element's address
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));

// scales that a whole wave shares, by scalar loads
typedef __attribute__((address_space(4))) float float_const;

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ring_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A block's partial sum, kept in program order; whoever reads it places the
// wait states.
__device__ __forceinline__ void mfma_start(v4f& p, const v8i& x, const v8i& y) {
  asm volatile("v_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, 0" : "=&v"(p) : "v"(x), "v"(y));
}

// A lane's number or address, in a form that the compiler cannot see through:
// what is derived from it is formed where it is used instead of ahead of the tile loop
// and held in registers across it.
__device__ __forceinline__ int opaque(int lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

__device__ __forceinline__ v8i fragment(const uint8_t* p, int sw) {
  return join(*reinterpret_cast<const v4i*>(p + sw), *reinterpret_cast<const v4i*>(p + (sw ^ 64)));
}

// ---- large tiles ------------------------------------------------------------
//
// WM x WN waves, two per SIMD, each with a TM x TN part of the tile in 16 x 16
// fragments.  LDS holds D blocks of 128 k of A and B (whole 128-byte lines of
// each row) and of A's scales, filled by direct global -> LDS copies; B's scale
// of a wave's columns, one of 128 x 128, is a scalar.
//
// A wave goes through a block column by column of fragments: FM MFMAs, each
// behind the 4 fmas that add the sum which its registers still hold (that of 4
// MFMAs before), times its row's scale, to the accumulators.  With the s_nop 18
// wait states lie between an MFMA and the fmas on its result.  The fmas run
// beside the MFMAs: a loop of both on registers reaches 3600 TFLOP/s on random
// codes, without the fmas 4200.  The fragments of B are read two columns ahead,
// those of A for the next block behind the last column's MFMAs.
//
// What bounds the loop is LDS: a block of 256 x 256 is 2048 cycles of MFMAs on each
// SIMD, for which the waves read 192 KB and the copies write 64 KB, at 128 bytes a
// cycle as many cycles; and a copy takes about 1.5 us to arrive with the chip full.
// A barrier behind the column before the last says
// that the next block has arrived.  Where D > 2 blocks fit, it also says that the
// block at hand has been read, and copies of D blocks later take its place.
// SPLIT (256 x 256, where D = 2): A's fragments are in registers from the
// start of a block on, and the first half of a wave's columns has been read in its
// middle.  A barrier there lets the copies of the block after the next go
// out: A and the first halves into the buffers that are left, the second halves
// into a third buffer.  8192 x 14336 x 4096 to bf16 takes 443 us so (2170 TFLOP/s; 470
// with the copies behind the one barrier); MFMAs and fmas alone 283, with the LDS
// reads 326, with the barriers 338, and with the copies 431 (of 8192 x 4096 x 14336).
//
// A workgroup takes tile after tile; the first blocks of the next tile are
// copied while the last ones of the present tile are multiplied, and the output
// goes through the last block's buffer.
template <int BM_, int BN_, int WM_, int WN_, int D_, bool SPLIT_ = false>
struct F8Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, D = D_;
  static constexpr bool SPLIT = SPLIT_;
  static constexpr int NW = WM * WN;                // waves
  static constexpr int TM = BM / WM, TN = BN / WN;  // a wave's part of the tile
  static constexpr int FM = TM / 16, FN = TN / 16;  // and its fragments
  static constexpr int CA = BM / 8 / NW, CB = BN / 8 / NW;  // 1 KiB copies of a wave and block
  static constexpr int COPIES = CA + CB + 1;
  static constexpr int LAG = FM >= 4 ? 1 : 4 / FM;  // columns between an MFMA and its fmas
  static constexpr int SZA = BM * 128, SZB = BN * 128, SZH = SZB / 2, SZS = BM * 4;
  // slot i of A (and in it the output's staging), of B, of B's second halves (SPLIT), of A's scales
  static constexpr int STEP_A = SPLIT ? SZA : SZA + SZB;
  static constexpr int OFF_B = SPLIT ? 2 * SZA : SZA, STEP_B = SPLIT ? SZH : SZA + SZB;
  static constexpr int OFF_H = 2 * SZA + 2 * SZH;
  static constexpr int OFF_S = SPLIT ? OFF_H + 3 * SZH : D * (SZA + SZB);
  static constexpr int LDS = OFF_S + D * SZS;
  static constexpr int PER_CU = LDS > 80 * 1024 ? 1 : 2;  // workgroups
  // column behind which copies are issued, over ISSUE columns; blocks in flight
  // behind the next one at the barrier before the last column
  static constexpr int FROM = SPLIT ? FN / 2 - 1 : FN - 2, ISSUE = SPLIT ? 3 : D > 2 ? 2 : 1;
  static constexpr int NEWER = SPLIT ? 1 : D - 2;
  static_assert(LDS <= 160 * 1024, "fits the 160 KiB LDS of a gfx950 CU");
  static_assert(CA * NW * 8 == BM && CB * NW * 8 == BN && NW % 2 == 0 && NW * 64 >= BM, "copies split evenly over the waves");
  static_assert(TN == 64 || TN == 128, "output staging; one scale of B for a wave");
  static_assert((SPLIT ? SZA : SZA + SZB) >= NW * 4096, "output staging");
  static_assert(!SPLIT || (D == 2 && NW == 8 && WN == 2 && TN == 128), "halves of B");
};

template <class T, bool GATHER>
struct F8Ring {
  static constexpr int FM = T::FM, FN = T::FN;

  static __device__ __forceinline__ void run(const F8Args& a, int tiles_n) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / T::WN, wn = wave % T::WN;
    const int g = lane >> 4, r = lane & 15;
    const int K = a.K, S = a.KB, tail = K & 127;

    // A copy moves 8 rows of 128 bytes: lane l fetches row l / 8, and of its
    // chunks the one that the swizzle puts at place l % 8 (the row's swizzle
    // depends on the parity of the copy's number, which is the wave's).
    constexpr int kRsrcWord3 = 0x00020000;
    // All of an offset is the lane's, so that the bounds check of the buffers (which
    // end with the tile's rows) sees it: rows past the tile's end read as zeros.
    const int c16 = ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 16;
    const uint32_t off0 = (uint32_t)((lane >> 3) * K + c16);
    __amdgpu_buffer_rsrc_t rs_a, rs_b, rs_s;
    const ExpertScan scan = scan_experts(a, T::BM, lane);
    auto find = [&](int64_t tile, ExpertTile& t) {
      if (!pick_tile(a, scan, T::BM, tiles_n, tile, opaque(threadIdx.x & 63), t)) return false;
      // as scalars
      t.row0 = __builtin_amdgcn_readfirstlane((int)t.row0);
      t.rows = __builtin_amdgcn_readfirstlane(t.rows);
      t.expert = __builtin_amdgcn_readfirstlane(t.expert);
      t.tn = __builtin_amdgcn_readfirstlane(t.tn);
      return true;
    };
    // what the copies of a tile read
    auto open = [&](const ExpertTile& t) {
      const int n0 = t.tn * T::BN, cols = min(T::BN, a.N - n0);
      if constexpr (GATHER) {
        rs_a = __builtin_amdgcn_make_buffer_rsrc((void*)a.A, 0, (int)(uint32_t)(a.rows_a * K), kRsrcWord3);
        rs_s = __builtin_amdgcn_make_buffer_rsrc((void*)a.SA, 0, (int)(uint32_t)(a.rows_a * S * 4), kRsrcWord3);
      } else {
        rs_a = __builtin_amdgcn_make_buffer_rsrc((void*)(a.A + t.row0 * K), 0, t.rows * K, kRsrcWord3);
        rs_s = __builtin_amdgcn_make_buffer_rsrc((void*)(a.SA + t.row0 * S), 0, t.rows * S * 4, kRsrcWord3);
      }
      rs_b = __builtin_amdgcn_make_buffer_rsrc((void*)(a.B + ((int64_t)t.expert * a.N + n0) * K), 0, cols * K,
                                               kRsrcWord3);
    };
    // Places in A and in its scales of the rows that this lane copies.  By index
    // they are looked up in two steps: the indices are loaded long before they
    // are needed.
    struct Rows {
      uint32_t a[GATHER ? T::CA : 1], s;
    };
    auto load_rows = [&](const ExpertTile& t) {
      Rows w;
      if constexpr (GATHER) {
        const int lane = opaque(threadIdx.x & 63);
        const int32_t* index = a.index + t.row0;
#pragma unroll
        for (int u = 0; u < T::CA; u++) w.a[u] = (uint32_t)index[min((wave + T::NW * u) * 8 + (lane >> 3), t.rows - 1)];
        w.s = (uint32_t)index[min((wave * 64 + lane) % T::BM, t.rows - 1)];
      }
      return w;
    };
    auto places = [&](Rows w) {
      if constexpr (GATHER) {
        const int lane = opaque(threadIdx.x & 63);
        const int c16 = ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 16;
        // a row outside A is read as row 0 (its results are NaN)
#pragma unroll
        for (int u = 0; u < T::CA; u++) w.a[u] = (uint32_t)(max(row_of_index(a, (int)w.a[u]), (int64_t)0) * K) + c16;
        w.s = (uint32_t)(max(row_of_index(a, (int)w.s), (int64_t)0) * S * 4);
      } else {
        w.a[0] = off0;
        w.s = (uint32_t)((wave * 64 + lane) % T::BM * S * 4);
      }
      return w;
    };
    // Slots of a block: `a` of D, and (SPLIT) `h` of 3 for the second halves of B.
    struct Slot {
      int a, h;
    };
    auto after = [&](Slot x) { return Slot{x.a + 1 == T::D ? 0 : x.a + 1, x.h == 2 ? 0 : x.h + 1}; };
    // the block D later
    auto later = [&](Slot x) { return Slot{x.a, x.h == 0 ? 2 : x.h - 1}; };
    // LDS place of this wave's copy v of B: rows 8 (wave + NW v)
    auto b_place = [&](Slot x, int v) {
      if (T::SPLIT) return ((v & 1) ? T::OFF_H + x.h * T::SZH : T::OFF_B + x.a * T::STEP_B) + ((v >> 1) * 8 + wave) * 1024;
      return T::OFF_B + x.a * T::STEP_B + (wave + T::NW * v) * 1024;
    };
    // and of column j of its fragments
    auto b_column = [&](Slot x, int j) {
      if (T::SPLIT)
        return (j >= FN / 2 ? T::OFF_H + x.h * T::SZH : T::OFF_B + x.a * T::STEP_B) + wn * (T::SZH / 2) +
               j % (FN / 2) * 2048;
      return T::OFF_B + x.a * T::STEP_B + wn * T::TN * 128 + j * 2048;
    };
    // copy u of COPIES of a block
    auto copy = [&](const Rows& w, int slice, Slot x, int u) {
      if (u < T::CA) {
        const int rows = (wave + T::NW * u) * 8;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, (lds_void*)(smem + x.a * T::STEP_A + rows * 128), 16,
                                                 w.a[GATHER ? u : 0] + (GATHER ? 0 : rows * K) + slice * 128, 0, 0, 0);
      } else if (u < T::CA + T::CB) {
        const int rows = (wave + T::NW * (u - T::CA)) * 8;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, (lds_void*)(smem + b_place(x, u - T::CA)), 16,
                                                 off0 + rows * K + slice * 128, 0, 0, 0);
      } else {
        // the scales of 64 rows (several waves bring the same ones)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_s, (lds_void*)(smem + T::OFF_S + x.a * T::SZS + (wave * 64 % T::BM) * 4),
                                                 4, w.s + slice * 4, 0, 0, 0);
      }
    };
    auto copy_all = [&](const Rows& w, int slice, Slot x) {
#pragma unroll
      for (int u = 0; u < T::COPIES; u++) copy(w, slice, x, u);
    };
    // In a partial last block the chunks past K that this lane fetched are other
    // rows' codes: zeros over A's and B's.
    auto zero_tail = [&](Slot x) {
      const int lane = opaque(threadIdx.x & 63);
      const int c16 = ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 16;
      if (c16 >= tail) {
#pragma unroll
        for (int u = 0; u < T::CA; u++)
          *reinterpret_cast<v4i*>(smem + x.a * T::STEP_A + (wave + T::NW * u) * 1024 + lane * 16) = v4i{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < T::CB; u++) *reinterpret_cast<v4i*>(smem + b_place(x, u) + lane * 16) = v4i{0, 0, 0, 0};
      }
    };

    int64_t tile = blockIdx.x;
    ExpertTile t;
    if (!find(tile, t)) return;
    // Copies cross from one tile to the next: block v of the present tile is
    // number v, block v of the next one number S + v.  (Not where a tile has fewer
    // blocks than LDS holds.)
    const bool cross = S >= T::D;
    bool first = true;
    Rows w = places(load_rows(t));
    Slot at = {0, 0};  // of the block at hand
    int ahead = 0;     // number of the last block whose copies are issued
    // lane address of a fragment's first half; the second half's is that with
    // bit 6 flipped, by the swizzle
    const int sw = r * 128 + ((g ^ ((r >> 1) & 7)) << 4);
    const int la = wm * T::TM * 128, ls = T::OFF_S + (wm * T::TM + r) * 4;

    for (;;) {
      if (!first) ring_barrier();  // the last tile's output is read back
      if (first || !cross) {
        open(t);
        if (!first) w = places(load_rows(t));
        Slot x = at;
        ahead = min(T::D, S) - 1;
        for (int i = 0; i <= ahead; i++) {
          copy_all(w, i, x);
          x = after(x);
        }
        if (S >= T::D)
          wait_vm<(T::D - 1) * T::COPIES>();
        else
          wait_vm<0>();
        if (tail != 0 && S == 1) zero_tail(at);
        ring_barrier();
      } else {
        // blocks 0 .. D - 2 are there since the last tile's output
        Slot x = at;
#pragma unroll
        for (int i = 1; i < T::D; i++) x = after(x);
        copy_all(w, T::D - 1, x);
        ahead = T::D - 1;
      }
      // columns past N (a wave may have no others) take the last block's scales
      const float_const* sb_at =
          (const float_const*)(a.SB + ((int64_t)t.expert * a.NB + min((t.tn * T::BN + wn * T::TN) >> 7, a.NB - 1)) * S);
      // the next tile, found here where few registers are in use
      ExpertTile following;
      Rows w_next;
      tile += gridDim.x;
      const bool next = find(tile, following);
      if (next) w_next = load_rows(following);
      v4f acc[FM][FN];
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++) acc[i][j] = v4f{0, 0, 0, 0};
      v8i fa[FM], fb[2];
      v4f p[T::LAG][FM];
      float sc[FM], sa[FM];  // scales of the sums at hand; A's of the block at hand
      float sb = sb_at[0];
#pragma unroll
      for (int f = 0; f < FM; f++) fa[f] = fragment(smem + at.a * T::STEP_A + la + f * 2048, sw);
      fb[0] = fragment(smem + b_column(at, 0), sw);
      fb[1] = fragment(smem + b_column(at, 1), sw);
#pragma unroll
      for (int f = 0; f < FM; f++) {
        sa[f] = *reinterpret_cast<const float*>(smem + ls + at.a * T::SZS + f * 64);
        sc[f] = 0.0f;
        // added with scale 0 ahead of the first columns
#pragma unroll
        for (int l = 0; l < T::LAG; l++) p[l][f] = v4f{0, 0, 0, 0};
      }
      for (int s = 0; s < S; s++) {
        // (what is read for a block past the last one is not used)
        const Slot then = after(at);
        float sb_next = sb_at[min(s + 1, S - 1)];
        int to_copy = -1;
#pragma unroll
        for (int j = 0; j < FN; j++) {
          const bool last = j == FN - 1;
          if (j == T::LAG) {
#pragma unroll
            for (int u = 0; u < FM; u++) sc[u] = sa[u] * sb;
          }
#pragma unroll
          for (int u = 0; u < FM; u++) {
            // the sums of the column LAG before; ahead of column LAG those of the block before
            v4f& c = acc[u][(j + FN - T::LAG) % FN];
            v4f& q = p[j % T::LAG][u];
            asm volatile("s_nop 2" : "+v"(q));
#pragma unroll
            for (int x = 0; x < 4; x++) c[x] = fmaf(q[x], sc[u], c[x]);
            asm volatile("" : "+v"(c));  // here, not behind the next branch
            __builtin_amdgcn_sched_barrier(0);
            mfma_start(q, fb[j & 1], fa[u]);
            if (last) fa[u] = fragment(smem + then.a * T::STEP_A + la + u * 2048, sw);
            __builtin_amdgcn_sched_barrier(0);
          }
          if (j == FN - 2) {
            // the next block is there (those that the tile starts with are since
            // the last tile's output; its stores are waited for with the copies
            // behind them)
            if (first || !cross || s + 2 >= T::D) {
              if (ahead - (s + 1) >= T::NEWER)
                wait_vm<T::NEWER * T::COPIES>();
              else
                wait_vm<0>();
            }
            if (tail != 0 && s + 2 == S) zero_tail(then);
            ring_barrier();
            asm volatile("" : "+s"(sb_next));  // loaded by now
          }
          // all have read what the copies take the place of
          if (T::SPLIT && j == T::FROM) asm volatile("s_barrier" ::: "memory");
          if (j == T::FROM) {
            const int v = s + T::D;
            if (v < S) {
              to_copy = v;
            } else if (cross && next && v < S + T::D - 1) {
              to_copy = v - S;
              if (v == S) {
                open(following);
                if (GATHER) w = places(w_next);
              }
            }
            if (to_copy >= 0) ahead = v;
          }
          if (j + 2 < FN)
            fb[j & 1] = fragment(smem + b_column(at, j + 2), sw);
          else
            fb[j & 1] = fragment(smem + b_column(then, j + 2 - FN), sw);
          const int part = j - T::FROM;
          if (part >= 0 && part < T::ISSUE && to_copy >= 0) {
#pragma unroll
            for (int u = part * T::COPIES / T::ISSUE; u < (part + 1) * T::COPIES / T::ISSUE; u++)
              copy(w, to_copy, later(at), u);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int u = 0; u < FM; u++) sa[u] = *reinterpret_cast<const float*>(smem + ls + then.a * T::SZS + u * 64);
        sb = sb_next;
        at = then;
      }
      asm volatile("s_nop 15\n\ts_nop 2" ::: "memory");
#pragma unroll
      for (int u = 0; u < FM; u++) {
#pragma unroll
        for (int l = 0; l < T::LAG; l++) {
          asm volatile("" : "+v"(p[l][u]));
          v4f& c = acc[u][FN - T::LAG + l];
#pragma unroll
          for (int x = 0; x < 4; x++) c[x] = fmaf(p[l][u][x], sc[u], c[x]);
        }
      }
      // the slot of the last block, which all have read
      uint8_t* cst = smem + (at.a == 0 ? T::D - 1 : at.a - 1) * T::STEP_A + wave * 4096;
      if (t.rows != T::BM || (t.tn + 1) * T::BN > a.N || (a.e.out != kOutF32 && joined(a))) {
        if (a.e.out == kOutF32)
          store<-1, 0>(a, t, acc, cst, wm, wn);
        else if (T::BN == 256 && joined(a))
          store16<-2, 0>(a, t, acc, cst, wm, wn);
        else
          store16<-1, 0>(a, t, acc, cst, wm, wn);
      } else if (a.e.act == kActGelu)
        store_typed<kActGelu>(a, t, acc, cst, wm, wn);
      else
        store_typed<kActNone>(a, t, acc, cst, wm, wn);
      if (!next) return;
      t = following;
      first = false;
    }
  }

  // Output: a lane holds 4 columns of row r of each fragment.  16 rows x 64
  // columns at a time go through 4 KiB of LDS and come back with consecutive
  // lanes on consecutive columns, so that the stores fill whole lines.
  // OUT >= 0: all rows and columns of the tile exist, and type and activation
  // are known here; OUT < 0: the general form.
  template <int OUT, int ACT>
  static __device__ __forceinline__ void store(const F8Args& a, const ExpertTile& t, v4f (&acc)[FM][FN], uint8_t* cst,
                                               int wm, int wn) {
    constexpr bool FULL = OUT >= 0;
    Epi e = a.e;
    if (FULL) {
      e.out = OUT;
      e.act = ACT;
    }
    const int lane = opaque(threadIdx.x & 63);
    const int rr = lane >> 4, cc = lane & 15;  // in a fragment: columns 4 rr, row cc; read back: row of 4, chunk
    const int64_t eb = (int64_t)t.expert * a.N;
    constexpr int NH = T::TN / 64;
    const int n0 = t.tn * T::BN + wn * T::TN + cc * 4;
    v4f bias[NH];
#pragma unroll
    for (int h = 0; h < NH; h++) {
      const int nc = n0 + h * 64;
      // -0 leaves every sum as it is
      bias[h] = v4f{-0.f, -0.f, -0.f, -0.f};
      if (a.e.bias != nullptr) {
        if (FULL)
          bias[h] = *reinterpret_cast<const v4f_any*>(a.e.bias + eb + nc);
        else
          bias[h] = load_columns(a.e.bias + eb, nc, a.N, 0.0f);
      }
    }
    bool out[FM];  // rows of A that do not exist
#pragma unroll
    for (int u = 0; u < FM; u++) {
      const int row = wm * T::TM + 16 * u + cc;
      out[u] = GATHER && (FULL || row < t.rows) && a_row(a, t.row0 + row) < 0;
    }
    // the next tile's first copies are older than these loads: none of them
    // is in flight behind this, and the stores are not waited for with them
    wait_vm<0>();
#pragma unroll
    for (int u = 0; u < FM; u++) {
#pragma unroll
      for (int h = 0; h < NH; h++) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          v4f v = acc[u][h * 4 + j];
          if (GATHER) {
#pragma unroll
            for (int x = 0; x < 4; x++) v[x] = out[u] ? __builtin_nanf("") : v[x];
          }
          *reinterpret_cast<v4f*>(cst + cc * 256 + (((j * 4 + rr) ^ cc) << 4)) = v;
        }
        wave_sync();
#pragma unroll FULL ? 4 : 1
        for (int q = 0; q < 4; q++) {
          const int br = q * 4 + rr;
          v4f v = *reinterpret_cast<const v4f*>(cst + br * 256 + ((cc ^ br) << 4));
          const int orow = wm * T::TM + 16 * u + br, nc = n0 + h * 64;
          if (FULL || (orow < t.rows && nc < a.N)) {
            v += bias[h];
            if (e.act == kActGelu) {
#pragma unroll
              for (int x = 0; x < 4; x++) v[x] = gelu(v[x]);
            }
            store_columns<true>(e, a.N, t.row0 + orow, nc, v);
          }
        }
        wave_sync();
      }
    }
  }

  // Where 16-bit rows do not start with half a line, the caches join the stores of the largest
  // tile to lines, in us joined / past them: 8000 x 2000 x 528 23.8 / 28.4 (128 x 128 26.7 /
  // 24.4), 8000 x 9992 x 528 106 / 116, 16384 x 4024 x 1040 119 / 127, 8192 x 9968 x 2064 216
  // / 231; even from results of 400 MB on (16384 x 20008 x 1040 645 / 646, x 20016 620 / 595).
  // Rows that start with half a line are joined by memory: 8000 x 9952 x 528 94.1 / 85.5,
  // 16384 x 20000 x 528 389 / 319, 8192 x 14368 x 2064 327 / 313.
  static __device__ __forceinline__ bool joined(const F8Args& a) { return T::BN == 256 && (a.N & 31) != 0; }

  // The same for 16-bit results: bias, activation and rounding first, so that 32 rows x
  // 64 columns go through the 4 KiB at once and come back 8 columns a lane (half the
  // LDS bytes, barriers and stores).  OUT = -2: the general form with joined stores.
  template <int OUT, int ACT>
  static __device__ __forceinline__ void store16(const F8Args& a, const ExpertTile& t, v4f (&acc)[FM][FN], uint8_t* cst,
                                                 int wm, int wn) {
    constexpr bool FULL = OUT >= 0;
    const bool bf16 = FULL ? OUT == kOutBF16 : a.e.out == kOutBF16, act = FULL ? ACT == kActGelu : a.e.act == kActGelu;
    const int lane = opaque(threadIdx.x & 63);
    const int rr = lane >> 4, cc = lane & 15;
    const int64_t eb = (int64_t)t.expert * a.N;
    const int n0 = t.tn * T::BN + wn * T::TN;
    bool out[FM];  // rows of A that do not exist
#pragma unroll
    for (int u = 0; u < FM; u++) {
      const int row = wm * T::TM + 16 * u + cc;
      out[u] = GATHER && (FULL || row < t.rows) && a_row(a, t.row0 + row) < 0;
    }
#pragma unroll
    for (int h = 0; h < T::TN / 64; h++) {
      v4f bias[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        // -0 leaves every sum as it is
        bias[j] = v4f{-0.f, -0.f, -0.f, -0.f};
        if (a.e.bias != nullptr) {
          const int n = n0 + h * 64 + j * 16 + rr * 4;
          if (FULL)
            bias[j] = *reinterpret_cast<const v4f_any*>(a.e.bias + eb + n);
          else
            bias[j] = load_columns(a.e.bias + eb, n, a.N, 0.0f);
        }
      }
      // the next tile's first copies are older than these loads: none of them
      // is in flight behind this, and the stores are not waited for with them
      if (h == 0) wait_vm<0>();
#pragma unroll
      for (int u0 = 0; u0 < FM; u0 += 2) {
#pragma unroll
        for (int u = u0; u < u0 + 2; u++) {
#pragma unroll
          for (int j = 0; j < 4; j++) {
            v4f v = acc[u][h * 4 + j] + bias[j];
            uint32_t b[4];
#pragma unroll
            for (int x = 0; x < 4; x++) {
              if (GATHER) v[x] = out[u] ? __builtin_nanf("") : v[x];
              if (act) v[x] = gelu(v[x]);
              // fp32 values first (no conversion fused with GELU's last product)
              if (OUT != kOutBF16) asm("" : "+v"(v[x]));
              b[x] = bf16 ? bf16_bits(v[x]) : f16_bits(v[x]);
            }
            const int chunk = 2 * j + (rr >> 1);
            *reinterpret_cast<v2i*>(cst + (u - u0) * 2048 + cc * 128 + ((chunk ^ (cc & 7)) << 4) + (rr & 1) * 8) =
                v2i{(int)(b[0] | (b[1] << 16)), (int)(b[2] | (b[3] << 16))};
          }
        }
        wave_sync();
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const int row = q * 8 + (lane >> 3), chunk = lane & 7;
          const v4i v = *reinterpret_cast<const v4i*>(cst + row * 128 + ((chunk ^ (row & 7)) << 4));
          const int64_t m = t.row0 + wm * T::TM + 16 * u0 + row;
          const int n = n0 + h * 64 + chunk * 8;
          uint16_t* const to = (uint16_t*)a.e.C + m * a.N + n;
          if (FULL || (wm * T::TM + 16 * u0 + row < t.rows && n + 8 <= a.N)) {
            if (OUT != -2)
              __builtin_nontemporal_store((v4i_any)v, reinterpret_cast<v4i_any*>(to));
            else
              *reinterpret_cast<v4i_any*>(to) = (v4i_any)v;
          } else if (wm * T::TM + 16 * u0 + row < t.rows) {
#pragma unroll
            for (int x = 0; x < 7; x++)
              if (n + x < a.N) to[x] = (uint16_t)(v[x >> 1] >> 16 * (x & 1));
          }
        }
        wave_sync();
      }
    }
  }

  template <int ACT>
  static __device__ __forceinline__ void store_typed(const F8Args& a, const ExpertTile& t, v4f (&acc)[FM][FN], uint8_t* cst,
                                                     int wm, int wn) {
    if (a.e.out == kOutF32)
      store<kOutF32, ACT>(a, t, acc, cst, wm, wn);
    else if (a.e.out == kOutBF16)
      store16<kOutBF16, ACT>(a, t, acc, cst, wm, wn);
    else
      store16<kOutF16, ACT>(a, t, acc, cst, wm, wn);
  }
};

template <class T, bool GATHER>
__global__ __launch_bounds__(T::NW * 64) __attribute__((amdgpu_waves_per_eu(2))) void fp8_ring_kernel(F8Args a,
                                                                                                     int tiles_n) {
  F8Ring<T, GATHER>::run(a, tiles_n);
}

template <class T>
hipError_t launch_ring(const F8Args& a, hipStream_t stream) {
  const int64_t tiles_n = (a.N + T::BN - 1) / T::BN;
  const int64_t tiles = tiles_n * expert_tiles_m(a, T::BM);
  if (tiles > 0x7fffffff) return hipErrorInvalidConfiguration;
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess) return e;
  const int64_t most = (int64_t)cus * T::PER_CU;
  const dim3 grid((unsigned)(tiles < most ? tiles : most)), block(T::NW * 64);
  if (a.index != nullptr)
    hipLaunchKernelGGL((fp8_ring_kernel<T, true>), grid, block, 0, stream, a, (int)tiles_n);
  else
    hipLaunchKernelGGL((fp8_ring_kernel<T, false>), grid, block, 0, stream, a, (int)tiles_n);
  return hipGetLastError();
}

// ---- few rows ---------------------------------------------------------------
//
// CW x KW waves on a tile of 16 MB rows x 16 CW columns: each wave has 16 of the
// columns and every KW-th block of 128 k (a line of each row).  A stage of LDS
// holds KW blocks, one for each group of waves, and each wave's copy of the
// scales of A for its block; D stages are in flight or in use, so that a CU
// keeps most of its LDS of memory requests going, which is what bounds such
// products (16 x 28672 x 8192: 235 MB in 39 us, 47.6 in changing calls through Python,
// 4.9 TB/s).  The groups' sums are added through LDS at the end.
template <int MB_, int CW_, int KW_, int D_>
struct F8Few {
  static constexpr int MB = MB_, CW = CW_, KW = KW_, D = D_;
  static constexpr int BM = 16 * MB, BN = 16 * CW, NW = CW * KW;
  static constexpr int PART = (BM + BN) * 128, OFF_S = KW * PART, STAGE = OFF_S + NW * 256, LDS = D * STAGE;
  // copies of 8 rows: RG for a block, NC for a stage, of which a wave issues
  // MIN or (the first REM waves) one more; and one of scales
  static constexpr int RG = (BM + BN) / 8, NC = RG * KW, MIN = NC / NW, REM = NC % NW, MAX = MIN + (REM ? 1 : 0);
  static constexpr int PER_CU = LDS > 80 * 1024 ? 1 : 2;  // workgroups
  static_assert(LDS <= 160 * 1024 && LDS >= NW * MB * 1024 && D >= 3, "stages, and the sums of all waves");
  static_assert(BM <= 64 && 128 % BN == 0, "a wave's scales; one scale of B for a tile");
};

template <class T, bool GATHER>
__global__ __launch_bounds__(T::NW * 64) void fp8_few_kernel(F8Args a, int tiles_n) {
  constexpr int MB = T::MB, CW = T::CW, KW = T::KW, NW = T::NW, D = T::D;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wave % CW, kw = wave / CW;
  const int g = lane >> 4, r = lane & 15;
  ExpertTile t;
  if (!find_tile(a, T::BM, tiles_n, (int64_t)blockIdx.y * gridDim.x + blockIdx.x, lane, t)) return;
  const int K = a.K, n0 = t.tn * T::BN, cols = min(T::BN, a.N - n0);
  const int S = a.KB, tail = K & 127;  // blocks
  const int I = (S + KW - 1) / KW;     // stages

  constexpr int kRsrcWord3 = 0x00020000;
  const auto rs_a = GATHER
                        ? __builtin_amdgcn_make_buffer_rsrc((void*)a.A, 0, (int)(uint32_t)(a.rows_a * K), kRsrcWord3)
                        : __builtin_amdgcn_make_buffer_rsrc((void*)(a.A + t.row0 * K), 0, t.rows * K, kRsrcWord3);
  const auto rs_s = GATHER
                        ? __builtin_amdgcn_make_buffer_rsrc((void*)a.SA, 0, (int)(uint32_t)(a.rows_a * S * 4), kRsrcWord3)
                        : __builtin_amdgcn_make_buffer_rsrc((void*)(a.SA + t.row0 * S), 0, t.rows * S * 4, kRsrcWord3);
  const auto rs_b = __builtin_amdgcn_make_buffer_rsrc((void*)(a.B + ((int64_t)t.expert * a.N + n0) * K), 0, cols * K,
                                                      kRsrcWord3);
  const float_const* sb_at = (const float_const*)(a.SB + ((int64_t)t.expert * a.NB + (n0 >> 7)) * S);
  // Copy u of this wave: rows 8 rg .. of block kp of the stage, A's rows first.
  // Rows past the end are fetched as the last one, rows outside A as row 0.
  auto source = [&](int row) -> int64_t {
    const int at = min(row, t.rows - 1);
    return GATHER ? max(a_row(a, t.row0 + at), (int64_t)0) : at;
  };
  uint32_t off[T::MAX];
#pragma unroll
  for (int u = 0; u < T::MAX; u++) {
    const int rg = (wave + NW * u) % T::RG;
    const int c16 = ((lane & 7) ^ (4 * (rg & 1) + (lane >> 4))) * 16;
    const int64_t row = rg < T::BM / 8 ? source(rg * 8 + (lane >> 3)) : min(rg * 8 - T::BM + (lane >> 3), cols - 1);
    off[u] = (uint32_t)(row * K) + c16;
  }
  const uint32_t off_s = (uint32_t)(source(lane % T::BM) * S * 4);
  auto issue = [&](int i, int stage) {
#pragma unroll
    for (int u = 0; u < T::MAX; u++) {
      const int q = wave + NW * u;
      if (u < T::MIN || wave < T::REM) {
        const int kp = q / T::RG, rg = q % T::RG;
        const int slice = min(i * KW + kp, S - 1);  // past K: not used
        uint32_t o = off[u];
        if (tail != 0 && slice == S - 1) {
          // chunks past K are fetched as the block's first one
          const int c16 = ((lane & 7) ^ (4 * (rg & 1) + (lane >> 4))) * 16;
          if (c16 >= tail) o -= c16;
        }
        lds_void* to = (lds_void*)(smem + stage * T::STAGE + kp * T::PART + rg * 1024);
        if (rg < T::BM / 8)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, to, 16, o, slice * 128, 0, 0);
        else
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, to, 16, o, slice * 128, 0, 0);
      }
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_s, (lds_void*)(smem + stage * T::STAGE + T::OFF_S + wave * 256), 4, off_s,
                                             min(i * KW + kw, S - 1) * 4, 0, 0);
  };
  v4f acc[MB];
#pragma unroll
  for (int i = 0; i < MB; i++) acc[i] = v4f{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < D - 1; i++)
    if (i < I) issue(i, i);
  const int sw = r * 128 + ((g ^ ((r >> 1) & 7)) << 4);
  int stage = 0;
  float sb = sb_at[min(kw, S - 1)];
  for (int i = 0; i < I; i++) {
    // this wave's copies of stage i are there, then everybody's; the stage
    // before has been read by all
    if (i + D - 2 >= I)
      wait_vm<0>();
    else if (wave < T::REM)
      wait_vm<(D - 2) * (T::MAX + 1)>();
    else
      wait_vm<(D - 2) * (T::MIN + 1)>();
    ring_barrier();
    if (i + D - 1 < I) issue(i + D - 1, stage == 0 ? D - 1 : stage - 1);
    const int slice = i * KW + kw;
    const float sb_next = sb_at[min(slice + KW, S - 1)];
    if (slice < S) {
      const uint8_t* pa = smem + stage * T::STAGE + kw * T::PART;
      const uint8_t* ps = smem + stage * T::STAGE + T::OFF_S + wave * 256 + r * 4;
      const v8i fb = fragment(pa + T::BM * 128 + cw * 2048, sw);
      // codes past K count as zeros
      const bool lo = tail == 0 || slice != S - 1 || g * 16 < tail, hi = tail == 0 || slice != S - 1 || 64 + g * 16 < tail;
#pragma unroll
      for (int u = 0; u < MB; u++) {
        v8i fa = fragment(pa + u * 2048, sw);
#pragma unroll
        for (int x = 0; x < 4; x++) {
          fa[x] = lo ? fa[x] : 0;
          fa[4 + x] = hi ? fa[4 + x] : 0;
        }
        const float s = *reinterpret_cast<const float*>(ps + u * 64) * sb;
        const v4f p = mfma_block(fb, fa);
#pragma unroll
        for (int x = 0; x < 4; x++) acc[u][x] = fmaf(p[x], s, acc[u][x]);
      }
    }
    sb = sb_next;
    stage = stage == D - 1 ? 0 : stage + 1;
  }
  // sums of the KW groups, a fragment per wave at a time
  constexpr int NF = MB * CW;
  v4f* part = reinterpret_cast<v4f*>(smem);  // [KW][NF][64]
  ring_barrier();
#pragma unroll
  for (int u = 0; u < MB; u++) part[(kw * NF + cw * MB + u) * 64 + lane] = acc[u];
  __syncthreads();
  for (int f = wave; f < NF; f += NW) {
    v4f sum = part[f * 64 + lane];
#pragma unroll
    for (int w = 1; w < KW; w++) sum += part[(w * NF + f) * 64 + lane];
    const int row = 16 * (f % MB) + r, n = n0 + 16 * (f / MB) + 4 * g;
    if (row < t.rows && n < a.N) {
      const int64_t m = t.row0 + row;
      if (GATHER && a_row(a, m) < 0) {
        const float nan = __builtin_nanf("");
        sum = v4f{nan, nan, nan, nan};
      }
      f8_store4<false>(a, t.expert, m, n, sum);
    }
  }
}

template <class T>
hipError_t launch_few(const F8Args& a, hipStream_t stream) {
  const int64_t tiles_n = (a.N + T::BN - 1) / T::BN;
  const int64_t tiles = tiles_n * expert_tiles_m(a, T::BM);
  if (tiles > 0x7fffffff) return hipErrorInvalidConfiguration;
  // in two dimensions: a launch has less than 2^32 threads in one
  const int64_t most = 1 << 20;
  const dim3 grid((unsigned)(tiles < most ? tiles : most), (unsigned)((tiles + most - 1) / most)), block(T::NW * 64);
  if (a.index != nullptr)
    hipLaunchKernelGGL((fp8_few_kernel<T, true>), grid, block, 0, stream, a, (int)tiles_n);
  else
    hipLaunchKernelGGL((fp8_few_kernel<T, false>), grid, block, 0, stream, a, (int)tiles_n);
  return hipGetLastError();
}

// ---- launch -----------------------------------------------------------------

// (16 x 16 with 5 stages leaves LDS for one workgroup a CU: the same time where there is a tile a
// CU, else 66 us instead of 51 for 16 x 28672 x 8192, 56 instead of 38 for 8 rows over 32 experts
// of 4096 x 4096)
using Tile16x16 = F8Few<1, 1, 4, 4>;
using Tile16x32 = F8Few<1, 2, 4, 3>;
using Tile32x32 = F8Few<2, 2, 4, 4>;
using Tile32x64 = F8Few<2, 4, 2, 3>;
using Tile128x128 = F8Cfg<128, 128, 2, 2, 2>;
// with a CU to itself: 8 waves, and two blocks more in flight
using Tile128x128Deep = F8Cfg<128, 128, 4, 2, 4>;
using Tile256x128 = F8Cfg<256, 128, 4, 2, 3>;
using Tile256x256 = F8Cfg<256, 256, 4, 2, 2, true>;
// where tiles of 128 x 128 are too few for all CUs
using Tile64x128 = F8Cfg<64, 128, 2, 2, 3>;

// variant V of kF8Variants
template <int V, class T>
hipError_t launch_variant(const F8Args& a, hipStream_t stream) {
  static_assert(T::BM == kF8Variants[V].bm && T::BN == kF8Variants[V].bn, "the variant's tile");
  static_assert(T::PER_CU == kF8Variants[V].per_cu, "workgroups that fit on a CU");
  if constexpr (V < 4)
    return launch_few<T>(a, stream);
  else
    return launch_ring<T>(a, stream);
}

hipError_t launch_gathered_far(const F8Args& a, hipStream_t stream) {
  const int64_t tiles_n = (a.N + kBN - 1) / kBN;
  const int64_t tiles = tiles_n * expert_tiles_m(a, kBM);
  if (tiles > 0x7fffffff) return hipErrorInvalidConfiguration;
  const int64_t most = (int64_t)kCus * 8;  // what runs at once takes tile after tile
  hipLaunchKernelGGL(fp8_tile_kernel, dim3((unsigned)(tiles < most ? tiles : most)), dim3(256), 0, stream, a,
                     (int)tiles_n);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8(const F8Args& args, hipStream_t stream) {
  F8Args a = args;
  set_division(a);
  // gathered rows are addressed by 32-bit offsets from A's start
  if (a.index != nullptr && a.rows_a * a.K >= ((int64_t)1 << 32)) return launch_gathered_far(a, stream);
  int v = f8_choice(a.M, a.N, a.K, a.offsets == nullptr ? 0 : a.E);
  switch (v) {
    case 0:
      return launch_variant<0, Tile16x16>(a, stream);
    case 1:
      return launch_variant<1, Tile16x32>(a, stream);
    case 2:
      return launch_variant<2, Tile32x32>(a, stream);
    case 3:
      return launch_variant<3, Tile32x64>(a, stream);
    case 4:
      return launch_variant<4, Tile128x128Deep>(a, stream);
    case 5:
      return launch_variant<5, Tile128x128>(a, stream);
    case 6:
      return launch_variant<6, Tile256x128>(a, stream);
    case 7:
      return launch_variant<7, Tile256x256>(a, stream);
    default:
      return launch_variant<8, Tile64x128>(a, stream);
  }
}

}  // namespace mxg
