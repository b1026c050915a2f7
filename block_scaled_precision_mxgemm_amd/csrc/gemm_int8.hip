// gemm_int8.hip - int8 x int8 products with one scale per token (row of A)
// and per output channel (row of B), dense and by expert:
//   C[i][j] = out(act(sa_i sb_j sum_k a_ik b_jk + bias_j)).
// The sum is exact: it stays in int32 (K < 2^17, so |sum| < 2^31 for any
// codes), and is rounded once, to fp32, before the scales.
//
// By expert, rows offsets[e] .. offsets[e+1] of C take B, its scales and its
// bias of expert e, and row p of C takes row index[p] / index_div of A (row p
// without an index).  The workgroups find their tile from the offsets on the
// device: no host copy of the row counts, and no work but a scan of them.
#include "int8_choice.h"
#include "mxg_int8.h"
#include "mxg_internal.h"

namespace mxg {
namespace {

// ---- gathered rows of an A of 4 GiB and more --------------------------------
//
// The one case that the kernels below, whose gathered rows are 32-bit offsets,
// do not take.  64 x 64 tiles, 4 waves of 32 x 32, slices of 128 k through
// registers.
constexpr int kBM = 64, kBN = 64, kBK = 128;

__global__ __launch_bounds__(256) void int8_tile_kernel(I8Args a, int tiles_n) {
  __shared__ __attribute__((aligned(16))) uint8_t sa[kBM * kBK], sb[kBN * kBK];
  __shared__ int64_t arow[kBM];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, r = lane & 15;
  I8Tile t;
  for (int64_t tile = blockIdx.x; find_tile(a, kBM, tiles_n, tile, lane, t); tile += gridDim.x) {
    __syncthreads();  // the rows of the tile before have been looked up by all
    if (tid < kBM) arow[tid] = tid < t.rows ? a_row(a, t.row0 + tid) : -1;
    __syncthreads();
    const int8_t* B = a.B + (int64_t)t.expert * a.N * a.K;
    const int n0 = t.tn * kBN;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    v4i acc[2][2] = {};
    for (int k0 = 0; k0 < a.K; k0 += kBK) {
      for (int c = tid; c < kBM * 8; c += 256) {
        const int row = c >> 3, ch = c & 7, k = k0 + ch * 16;
        const int64_t ar = arow[row];
        v4i va = {0, 0, 0, 0}, vb = {0, 0, 0, 0};
        if (ar >= 0 && k < a.K) va = *reinterpret_cast<const v4i*>(a.A + ar * a.K + k);
        if (n0 + row < a.N && k < a.K) vb = *reinterpret_cast<const v4i*>(B + (int64_t)(n0 + row) * a.K + k);
        const int o = row * kBK + ((ch ^ swz8(row)) << 4);
        *reinterpret_cast<v4i*>(sa + o) = va;
        *reinterpret_cast<v4i*>(sb + o) = vb;
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; h++) {
        v4i fa[2], fb[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const int ra = wm + 16 * i + r, rb = wn + 16 * i + r;
          fa[i] = *reinterpret_cast<const v4i*>(sa + ra * kBK + (((4 * h + g) ^ swz8(ra)) << 4));
          fb[i] = *reinterpret_cast<const v4i*>(sb + rb * kBK + (((4 * h + g) ^ swz8(rb)) << 4));
        }
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
          for (int j = 0; j < 2; j++) acc[i][j] = mfma_i8(fb[j], fa[i], acc[i][j]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int row = wm + 16 * i + r;
      if (row >= t.rows) continue;
      const float s = a_scale(a, arow[row]);
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const int n = n0 + wn + 16 * j + 4 * g;
        if (n < a.N) store4(a, t.expert, t.row0 + row, n, acc[i][j], s);
      }
    }
  }
}

// ---- large tiles ------------------------------------------------------------
//
// WM x WN waves, two per SIMD, each with a TM x TN part of the tile in 16 x 16
// fragments.  K goes by slices of 128 (whole 128-byte lines of each row) in
// two steps of 64; LDS holds DB slices of B and one more of A, filled by direct
// global -> LDS copies.  While a wave runs the MFMAs of one step on registers
// it reads the fragments of the next step from LDS, so only one barrier per
// slice is needed: behind the first step's MFMAs, when slice s has been read
// by all and slice s + 1 has arrived.  The copies of slice s + DB are spread over
// the steps, so that their issue does not hold up the MFMAs: B's behind the
// barrier, into the buffer that slice s left, A's (into the buffer of slice
// s - 1) in the step before.
//
// A workgroup takes tile after tile; the first copies of the next tile are
// issued before the last step of the present one, and its output goes through
// the last A buffer, which those copies leave alone.
template <int BM_, int BN_, int WM_, int WN_, int DB_ = 2>
struct I8Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int DB = DB_, DA = DB + 1;       // slices of B and of A in LDS
  static constexpr int NW = WM * WN;                // waves
  static constexpr int TM = BM / WM, TN = BN / WN;  // a wave's part of the tile
  static constexpr int FM = TM / 16, FN = TN / 16;  // and its fragments
  static constexpr int CA = BM / 8 / NW, CB = BN / 8 / NW;  // 1 KiB copies of a wave and slice
  static constexpr int SZA = BM * 128, SZB = BN * 128;
  static constexpr int OFF_B = DA * SZA;
  // output staging, 4 KiB per wave: the last A buffer, or its own
  static constexpr bool OWN = SZA < NW * 4096;
  static constexpr int OFF_CST = OWN ? OFF_B + DB * SZB : DB * SZA;
  static constexpr int LDS = OFF_B + DB * SZB + (OWN ? NW * 4096 : 0);
  // copies issued after slice s + 1's when it is waited for in slice s
  static constexpr int NEWER = (DB - 2) * (CA + CB) + CA;
  static constexpr int PER_CU = LDS > 80 * 1024 ? 1 : LDS > 40 * 1024 ? 2 : 4;  // workgroups
  static_assert(LDS <= 160 * 1024, "fits the 160 KiB LDS of a gfx950 CU");
  static_assert(CA * NW * 8 == BM && CB * NW * 8 == BN && NW % 2 == 0, "copies split evenly over the waves");
  static_assert(TN % 64 == 0, "output staging");
};

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ring_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// int8 MFMA with the accumulator tied in place in AGPRs, kept in program order:
// left to itself the compiler moves fragments through AGPRs.
__device__ __forceinline__ void i8_mfma_acc(v4i& c, const v4i& x, const v4i& y) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(x), "v"(y));
}
// wait states around the inline MFMAs, as mfma_fence_init and mfma_drain
template <int NI, int NJ>
__device__ __forceinline__ void i8_fence_init(v4i (&acc)[NI][NJ]) {
#pragma unroll
  for (int i = 0; i < NI; i++)
#pragma unroll
    for (int j = 0; j < NJ; j++) asm volatile("" : "+a"(acc[i][j]));
  asm volatile("s_nop 7" ::: "memory");
}
template <int NI, int NJ>
__device__ __forceinline__ void i8_drain(v4i (&acc)[NI][NJ]) {
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int i = 0; i < NI; i++)
#pragma unroll
    for (int j = 0; j < NJ; j++) asm volatile("" : "+a"(acc[i][j]));
}

// A lane's number or address, in a form that the compiler cannot see through:
// what is derived from it is formed where it is used instead of ahead of the tile loop
// and held in registers across it.
__device__ __forceinline__ int opaque(int lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

template <class T, bool GATHER>
struct RingKernel {
  static constexpr int FM = T::FM, FN = T::FN;

  // MFMAs of a step, column by column of fragments, on the rows' fragments
  // `ca` and the columns' `fb`; `also(j)` runs behind column j.  From the
  // second column on the fragments of the next step are read: a column's into
  // the registers that its MFMAs have left, the rows' into `na`.
  template <class F>
  static __device__ __forceinline__ void step(v4i (&acc)[FM][FN], const v4i (&ca)[FM], v4i (&na)[FM], v4i (&fb)[FN],
                                              const uint8_t* ra, const uint8_t* rb, F also) {
#pragma unroll
    for (int j = 0; j < FN; j++) {
#pragma unroll
      for (int u = 0; u < FM; u++) i8_mfma_acc(acc[u][j], fb[j], ca[u]);
      __builtin_amdgcn_sched_barrier(0);
      also(j);
      if (j >= 1) {
#pragma unroll
        for (int u = 0; u < FM; u++)
          if (u * (FN - 1) / FM == j - 1) na[u] = *reinterpret_cast<const v4i*>(ra + u * 2048);
        if (j == 1) fb[0] = *reinterpret_cast<const v4i*>(rb);
        fb[j] = *reinterpret_cast<const v4i*>(rb + j * 2048);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  static __device__ __forceinline__ void run(const I8Args& a, int tiles_n) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / T::WN, wn = wave % T::WN;
    const int g = lane >> 4, r = lane & 15;
    const int K = a.K;
    const int S = (K + 127) >> 7, tail = K & 127;

    // A copy moves 8 rows of 128 bytes: lane l fetches row l / 8, and of its
    // chunks the one that the swizzle puts at place l % 8 (the row's swizzle
    // depends on the parity of the copy's number, which is the wave's).
    constexpr int kRsrcWord3 = 0x00020000;
    const int c16 = ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 16;
    const uint32_t off0 = (uint32_t)((8 * wave + (lane >> 3)) * K + c16);
    const uint32_t rows_step = (uint32_t)(8 * T::NW * K);
    I8Tile t;
    __amdgpu_buffer_rsrc_t rs_a, rs_b;
    uint32_t oa[GATHER ? T::CA : 1], lim_a = 0, lim_b = 0;
    auto set_tile = [&](int64_t tile) -> bool {
      const int lane = opaque(threadIdx.x & 63);
      const int c16 = ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 16;
      if (!find_tile(a, T::BM, tiles_n, tile, lane, t)) return false;
      const int n0 = t.tn * T::BN, cols = min(T::BN, a.N - n0);
      if constexpr (GATHER) {
#pragma unroll
        for (int u = 0; u < T::CA; u++) {
          const int row = min((wave + T::NW * u) * 8 + (lane >> 3), t.rows - 1);
          // a row outside A is read as row 0 (its results are NaN)
          oa[u] = (uint32_t)(max(a_row(a, t.row0 + row), (int64_t)0) * K) + c16;
        }
        rs_a = __builtin_amdgcn_make_buffer_rsrc((void*)a.A, 0, (int)(uint32_t)(a.rows_a * K), kRsrcWord3);
      } else {
        lim_a = (uint32_t)((t.rows - 1) * K + c16);
        rs_a = __builtin_amdgcn_make_buffer_rsrc((void*)(a.A + t.row0 * K), 0, t.rows * K, kRsrcWord3);
      }
      lim_b = (uint32_t)((cols - 1) * K + c16);
      rs_b = __builtin_amdgcn_make_buffer_rsrc((void*)(a.B + ((int64_t)t.expert * a.N + n0) * K), 0, cols * K,
                                               kRsrcWord3);
      return true;
    };
    // Rows past the tile's are fetched as its last one; in a partial last
    // slice, chunks past K as the slice's first one.
    auto back = [&](int slice) {
      const int lane = opaque(threadIdx.x & 63);
      const int c16 = ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 16;
      return (tail != 0 && slice == S - 1 && c16 >= tail) ? (uint32_t)c16 : 0u;
    };
    auto copy_a1 = [&](int slice, int buf, uint32_t b, int u) {
      const uint32_t o = GATHER ? oa[GATHER ? u : 0] : min(off0 + u * rows_step, lim_a);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, (lds_void*)(smem + buf * T::SZA + (wave + T::NW * u) * 1024), 16,
                                               o - b, slice * 128, 0, 0);
    };
    auto copy_b1 = [&](int slice, int buf, uint32_t b, int u) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs_b, (lds_void*)(smem + T::OFF_B + buf * T::SZB + (wave + T::NW * u) * 1024), 16,
          min(off0 + u * rows_step, lim_b) - b, slice * 128, 0, 0);
    };
    auto copy_a = [&](int slice, int buf, uint32_t b) {
#pragma unroll
      for (int u = 0; u < T::CA; u++) copy_a1(slice, buf, b, u);
    };
    auto copy_b = [&](int slice, int buf, uint32_t b) {
#pragma unroll
      for (int u = 0; u < T::CB; u++) copy_b1(slice, buf, b, u);
    };
    // zeros over the chunks of A past K that this lane fetched (their
    // products vanish whatever B's are)
    auto zero_tail = [&](int buf) {
      const int lane = opaque(threadIdx.x & 63);
      const int c16 = ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 16;
      if (c16 >= tail) {
#pragma unroll
        for (int u = 0; u < T::CA; u++)
          *reinterpret_cast<v4i*>(smem + buf * T::SZA + (wave + T::NW * u) * 1024 + lane * 16) = v4i{0, 0, 0, 0};
      }
    };
    auto start_tile = [&]() {
#pragma unroll
      for (int i = 0; i < T::DB; i++)
        if (i < S) {
          copy_a(i, i, back(i));
          copy_b(i, i, back(i));
        }
    };

    int64_t tile = blockIdx.x;
    if (!set_tile(tile)) return;
    start_tile();
    bool first = true;
    if (S >= T::DB)
      wait_vm<(T::DB - 1) * (T::CA + T::CB)>();
    else
      wait_vm<0>();
    // lane addresses of a slice's first step (of A's and B's rows); the second
    // step's are those with bit 6 flipped, by the swizzle
    const int sw0 = r * 128 + ((g ^ ((r >> 1) & 7)) << 4);
    const int la = wm * T::TM * 128, lb = T::OFF_B + wn * T::TN * 128;

    for (;;) {
      // this wave's copies of slice 0 are there (and the last tile's output is
      // read back)
      if (tail != 0 && S == 1) zero_tail(0);
      ring_barrier();
      v4i acc[FM][FN];
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++) acc[i][j] = v4i{0, 0, 0, 0};
      i8_fence_init(acc);
      v4i a0[FM], a1[FM], fb[FN];
      {
        const int lane = opaque(threadIdx.x & 63), g = lane >> 4, r = lane & 15;
        const uint8_t* first = smem + r * 128 + ((g ^ ((r >> 1) & 7)) << 4);
#pragma unroll
        for (int f = 0; f < FM; f++) a0[f] = *reinterpret_cast<const v4i*>(first + la + f * 2048);
#pragma unroll
        for (int f = 0; f < FN; f++) fb[f] = *reinterpret_cast<const v4i*>(first + lb + f * 2048);
      }
      const I8Tile now = t;
      bool next = false;
      int ba = 0, bb = 0, s = 0;  // buffers of slice s
      // Slices that the tile started with are there since then, except in the
      // first tile; the last tile's stores are waited for with the copies that
      // follow them.
      for (; s + T::DB + 1 < S; s++) {
        const int an = ba == T::DB ? 0 : ba + 1, ap = ba == 0 ? T::DB : ba - 1;
        const int bn = bb == T::DB - 1 ? 0 : bb + 1;
        // A's slice s + DB, into the buffer of slice s - 1
        step(acc, a0, a1, fb, smem + ba * T::SZA + la + (sw0 ^ 64), smem + bb * T::SZB + lb + (sw0 ^ 64), [&](int j) {
#pragma unroll
          for (int u = 0; u < T::CA; u++)
            if ((u * FN) / T::CA == j) copy_a1(s + T::DB, ap, 0, u);
        });
        step(acc, a1, a0, fb, smem + an * T::SZA + la + sw0, smem + bn * T::SZB + lb + sw0, [&](int j) {
          if (j == 1) {
            if (first || s >= T::DB - 1) wait_vm<T::NEWER>();
            ring_barrier();
          }
#pragma unroll
          for (int u = 0; u < T::CB; u++)
            if (j >= 1 && 1 + (u * (FN - 1)) / T::CB == j) copy_b1(s + T::DB, bb, 0, u);
        });
        ba = an;
        bb = bn;
      }
      // the last slices: less and less is left to copy
      for (; s < S; s++) {
        const int an = ba == T::DB ? 0 : ba + 1, ap = ba == 0 ? T::DB : ba - 1;
        const int bn = bb == T::DB - 1 ? 0 : bb + 1;
        const bool more = s + T::DB < S;
        if (more) copy_a(s + T::DB, ap, back(s + T::DB));
        step(acc, a0, a1, fb, smem + ba * T::SZA + la + (sw0 ^ 64), smem + bb * T::SZB + lb + (sw0 ^ 64), [](int) {});
        step(acc, a1, a0, fb, smem + an * T::SZA + la + sw0, smem + bn * T::SZB + lb + sw0, [&](int j) {
          if (j != 1) return;
          if (first || s >= T::DB - 1) {
            if (more)
              wait_vm<T::NEWER>();
            else
              wait_vm<0>();
          }
          if (tail != 0 && s + 2 == S) zero_tail(an);
          ring_barrier();
          if (more) copy_b(s + T::DB, bb, back(s + T::DB));
          if (s + 1 == S) {
            tile += gridDim.x;
            next = set_tile(tile);
            if (next) start_tile();
          }
        });
        ba = an;
        bb = bn;
      }
      first = false;
      i8_drain(acc);
      uint8_t* cst = smem + T::OFF_CST + wave * 4096;
      if (now.rows != T::BM || (now.tn + 1) * T::BN > a.N)
        store<-1, 0>(a, now, acc, cst, wm, wn);
      else if (a.e.act == kActGelu)
        store_typed<kActGelu>(a, now, acc, cst, wm, wn);
      else
        store_typed<kActNone>(a, now, acc, cst, wm, wn);
      if (!next) return;
    }
  }

  // Output: a lane holds 4 columns of row r of each fragment.  16 rows x 64
  // columns at a time go through 4 KiB of LDS and come back with consecutive
  // lanes on consecutive columns, so that the stores fill whole lines.
  // OUT >= 0: all rows and columns of the tile exist, and type and activation are known here, so that what is run is short (each
  // tile fetches it anew); OUT < 0: the general form.
  template <int OUT, int ACT>
  static __device__ __forceinline__ void store(const I8Args& a, const I8Tile& t, v4i (&acc)[FM][FN], uint8_t* cst,
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
    v4f sb[NH], bias[NH];
#pragma unroll
    for (int h = 0; h < NH; h++) {
      const int nc = n0 + h * 64;
      // -0 leaves every sum as it is
      bias[h] = v4f{-0.f, -0.f, -0.f, -0.f};
      if (FULL) {
        sb[h] = *reinterpret_cast<const v4f_any*>(a.SB + eb + nc);
        if (a.e.bias != nullptr) bias[h] = *reinterpret_cast<const v4f_any*>(a.e.bias + eb + nc);
      } else {
        sb[h] = load_columns(a.SB + eb, nc, a.N, 0.0f);
        if (a.e.bias != nullptr) bias[h] = load_columns(a.e.bias + eb, nc, a.N, 0.0f);
      }
    }
    float sa[FM];
#pragma unroll
    for (int u = 0; u < FM; u++) {
      const int row = wm * T::TM + 16 * u + cc;
      sa[u] = FULL || row < t.rows ? a_scale(a, GATHER ? a_row(a, t.row0 + row) : t.row0 + row) : 0.0f;
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
          v4f v;
#pragma unroll
          for (int x = 0; x < 4; x++) v[x] = rounded_product((float)acc[u][h * 4 + j][x], sa[u]);
          *reinterpret_cast<v4f*>(cst + cc * 256 + (((j * 4 + rr) ^ cc) << 4)) = v;
        }
        wave_sync();
#pragma unroll FULL ? 4 : 1
        for (int q = 0; q < 4; q++) {
          const int br = q * 4 + rr;
          v4f v = *reinterpret_cast<const v4f*>(cst + br * 256 + ((cc ^ br) << 4));
          const int orow = wm * T::TM + 16 * u + br, nc = n0 + h * 64;
          if (FULL || (orow < t.rows && nc < a.N)) {
#pragma unroll
            for (int x = 0; x < 4; x++) v[x] = rounded_product(v[x], sb[h][x]) + bias[h][x];
            if (e.act == kActGelu) {
#pragma unroll
              for (int x = 0; x < 4; x++) v[x] = gelu(v[x]);
            }
            if constexpr (OUT == kOutF16) {
              // fp32 values first, as where the type is not known: else the
              // compiler makes one instruction of GELU's last product and the
              // conversion (v_fma_mixlo_f16, one rounding instead of two)
#pragma unroll
              for (int x = 0; x < 4; x++) asm("" : "+v"(v[x]));
            }
            store_columns<true>(e, a.N, t.row0 + orow, nc, v);
          }
        }
        wave_sync();
      }
    }
  }

  template <int ACT>
  static __device__ __forceinline__ void store_typed(const I8Args& a, const I8Tile& t, v4i (&acc)[FM][FN], uint8_t* cst,
                                                     int wm, int wn) {
    if (a.e.out == kOutF32)
      store<kOutF32, ACT>(a, t, acc, cst, wm, wn);
    else if (a.e.out == kOutBF16)
      store<kOutBF16, ACT>(a, t, acc, cst, wm, wn);
    else
      store<kOutF16, ACT>(a, t, acc, cst, wm, wn);
  }
};

template <class T, bool GATHER>
__global__ __launch_bounds__(T::NW * 64) __attribute__((amdgpu_waves_per_eu(2))) void int8_ring_kernel(I8Args a,
                                                                                                      int tiles_n) {
  RingKernel<T, GATHER>::run(a, tiles_n);
}

template <class T>
hipError_t launch_ring(const I8Args& a, hipStream_t stream) {
  const int64_t tiles_n = (a.N + T::BN - 1) / T::BN;
  const int64_t tiles = tiles_n * i8_tiles_m(a, T::BM);
  if (tiles > 0x7fffffff) return hipErrorInvalidConfiguration;
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess) return e;
  const int64_t most = (int64_t)cus * T::PER_CU;
  const dim3 grid((unsigned)(tiles < most ? tiles : most)), block(T::NW * 64);
  if (a.index != nullptr)
    hipLaunchKernelGGL((int8_ring_kernel<T, true>), grid, block, 0, stream, a, (int)tiles_n);
  else
    hipLaunchKernelGGL((int8_ring_kernel<T, false>), grid, block, 0, stream, a, (int)tiles_n);
  return hipGetLastError();
}

// ---- few rows ---------------------------------------------------------------
//
// CW x KW waves on a tile of 16 MB rows x 16 CW columns: each wave has 16 of the
// columns and every KW-th slice of 128 k (a line of each row).  A stage
// of LDS holds KW slices, one for each group of waves; D stages are in flight
// or in use, so that a CU keeps most of its LDS of memory requests going, which
// is what bounds such products.  The groups' sums are exact and are added
// through LDS at the end.
template <int MB_, int CW_, int KW_, int D_>
struct I8Few {
  static constexpr int MB = MB_, CW = CW_, KW = KW_, D = D_;
  static constexpr int BM = 16 * MB, BN = 16 * CW, NW = CW * KW;
  static constexpr int PART = (BM + BN) * 128, STAGE = KW * PART, LDS = D * STAGE;
  // copies of 8 rows: RG for a slice, NC for a stage, of which a wave issues
  // MIN or (the first REM waves) one more
  static constexpr int RG = (BM + BN) / 8, NC = RG * KW, MIN = NC / NW, REM = NC % NW, MAX = MIN + (REM ? 1 : 0);
  static_assert(LDS <= 160 * 1024 && LDS >= NW * MB * 1024 && D >= 3, "stages, and the sums of all waves");
};

template <class T, bool GATHER>
__global__ __launch_bounds__(T::NW * 64) void int8_few_kernel(I8Args a, int tiles_n) {
  constexpr int MB = T::MB, CW = T::CW, KW = T::KW, NW = T::NW, D = T::D;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wave % CW, kw = wave / CW;
  const int g = lane >> 4, r = lane & 15;
  I8Tile t;
  if (!find_tile(a, T::BM, tiles_n, blockIdx.x, lane, t)) return;
  const int K = a.K, n0 = t.tn * T::BN, cols = min(T::BN, a.N - n0);
  const int S = (K + 127) >> 7, tail = K & 127;  // slices
  const int I = (S + KW - 1) / KW;               // stages

  constexpr int kRsrcWord3 = 0x00020000;
  const auto rs_a = GATHER
                        ? __builtin_amdgcn_make_buffer_rsrc((void*)a.A, 0, (int)(uint32_t)(a.rows_a * K), kRsrcWord3)
                        : __builtin_amdgcn_make_buffer_rsrc((void*)(a.A + t.row0 * K), 0, t.rows * K, kRsrcWord3);
  const auto rs_b = __builtin_amdgcn_make_buffer_rsrc((void*)(a.B + ((int64_t)t.expert * a.N + n0) * K), 0, cols * K,
                                                      kRsrcWord3);
  // Copy u of this wave: rows 8 rg .. of slice kp of the stage, A's rows first.
  // Rows past the end are fetched as the last one, rows outside A as row 0.
  uint32_t off[T::MAX];
#pragma unroll
  for (int u = 0; u < T::MAX; u++) {
    const int rg = (wave + NW * u) % T::RG;
    const int c16 = ((lane & 7) ^ (4 * (rg & 1) + (lane >> 4))) * 16;
    int64_t row;
    if (rg < T::BM / 8) {
      row = min(rg * 8 + (lane >> 3), t.rows - 1);
      if (GATHER) row = max(a_row(a, t.row0 + row), (int64_t)0);
    } else {
      row = min(rg * 8 - T::BM + (lane >> 3), cols - 1);
    }
    off[u] = (uint32_t)(row * K) + c16;
  }
  auto issue = [&](int i, int stage) {
#pragma unroll
    for (int u = 0; u < T::MAX; u++) {
      const int q = wave + NW * u;
      if (u < T::MIN || wave < T::REM) {
        const int kp = q / T::RG, rg = q % T::RG;
        const int slice = min(i * KW + kp, S - 1);  // past K: not used
        uint32_t o = off[u];
        if (tail != 0 && slice == S - 1) {
          // chunks past K are fetched as the slice's first one
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
  };
  v4i acc[MB];
#pragma unroll
  for (int i = 0; i < MB; i++) acc[i] = v4i{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < D - 1; i++)
    if (i < I) issue(i, i);
  const int sw0 = r * 128 + ((g ^ ((r >> 1) & 7)) << 4);
  int stage = 0;
  for (int i = 0; i < I; i++) {
    // this wave's copies of stage i are there, then everybody's; the stage
    // before has been read by all
    if (i + D - 2 >= I)
      wait_vm<0>();
    else if (wave < T::REM)
      wait_vm<(D - 2) * T::MAX>();
    else
      wait_vm<(D - 2) * T::MIN>();
    ring_barrier();
    if (i + D - 1 < I) issue(i + D - 1, stage == 0 ? D - 1 : stage - 1);
    const int slice = i * KW + kw;
    if (slice < S) {
      const uint8_t* pa = smem + stage * T::STAGE + kw * T::PART;
      const uint8_t* pb = pa + T::BM * 128 + cw * 2048;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int sw = sw0 ^ (64 * h);
        v4i fa[MB];
#pragma unroll
        for (int u = 0; u < MB; u++) fa[u] = *reinterpret_cast<const v4i*>(pa + u * 2048 + sw);
        const v4i fb = *reinterpret_cast<const v4i*>(pb + sw);
        // codes past K count as zeros
        if (tail != 0 && slice == S - 1 && h * 64 + g * 16 >= tail) {
#pragma unroll
          for (int u = 0; u < MB; u++) fa[u] = v4i{0, 0, 0, 0};
        }
#pragma unroll
        for (int u = 0; u < MB; u++) acc[u] = mfma_i8(fb, fa[u], acc[u]);
      }
    }
    stage = stage == D - 1 ? 0 : stage + 1;
  }
  // sums of the KW groups, a fragment per wave at a time
  constexpr int NF = MB * CW;
  v4i* part = reinterpret_cast<v4i*>(smem);  // [KW][NF][64]
  ring_barrier();
#pragma unroll
  for (int u = 0; u < MB; u++) part[(kw * NF + cw * MB + u) * 64 + lane] = acc[u];
  __syncthreads();
  for (int f = wave; f < NF; f += NW) {
    v4i sum = part[f * 64 + lane];
#pragma unroll
    for (int w = 1; w < KW; w++) sum += part[(w * NF + f) * 64 + lane];
    const int row = 16 * (f % MB) + r, n = n0 + 16 * (f / MB) + 4 * g;
    if (row < t.rows && n < a.N) {
      const int64_t m = t.row0 + row;
      store4(a, t.expert, m, n, sum, a_scale(a, GATHER ? a_row(a, m) : m));
    }
  }
}

template <class T>
hipError_t launch_few(const I8Args& a, hipStream_t stream) {
  const int64_t tiles_n = (a.N + T::BN - 1) / T::BN;
  const int64_t tiles = tiles_n * i8_tiles_m(a, T::BM);
  if (tiles > 0x7fffffff) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)tiles), block(T::NW * 64);
  if (a.index != nullptr)
    hipLaunchKernelGGL((int8_few_kernel<T, true>), grid, block, 0, stream, a, (int)tiles_n);
  else
    hipLaunchKernelGGL((int8_few_kernel<T, false>), grid, block, 0, stream, a, (int)tiles_n);
  return hipGetLastError();
}

// ---- launch -----------------------------------------------------------------

using Tile16x16 = I8Few<1, 1, 4, 5>;
using Tile16x32 = I8Few<1, 2, 4, 3>;
using Tile32x32 = I8Few<2, 2, 4, 4>;
using Tile32x64 = I8Few<2, 4, 2, 3>;
using Tile128x128 = I8Cfg<128, 128, 2, 2>;
// with a CU to itself: 8 waves, as one wave alone cannot issue 16 x 16 MFMAs at
// the rate that the matrix core takes them, and a slice more in flight
using Tile128x128Deep = I8Cfg<128, 128, 4, 2, 3>;
using Tile256x128 = I8Cfg<256, 128, 4, 2>;
using Tile256x256 = I8Cfg<256, 256, 4, 2>;

// variant V of kI8Variants
template <int V, class T>
hipError_t launch_variant(const I8Args& a, hipStream_t stream) {
  static_assert(T::BM == kI8Variants[V].bm && T::BN == kI8Variants[V].bn, "the variant's tile");
  if constexpr (V < 4)
    return launch_few<T>(a, stream);
  else
    return launch_ring<T>(a, stream);
}

hipError_t launch_gathered_far(const I8Args& a, hipStream_t stream) {
  const int64_t tiles_n = (a.N + kBN - 1) / kBN;
  const int64_t tiles = tiles_n * i8_tiles_m(a, kBM);
  if (tiles > 0x7fffffff) return hipErrorInvalidConfiguration;
  const int64_t most = (int64_t)kCus * 8;  // what runs at once takes tile after tile
  hipLaunchKernelGGL(int8_tile_kernel, dim3((unsigned)(tiles < most ? tiles : most)), dim3(256), 0, stream, a,
                     (int)tiles_n);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8(const I8Args& args, hipStream_t stream) {
  I8Args a = args;
  set_division(a);
  // gathered rows are addressed by 32-bit offsets from A's start
  if (a.index != nullptr && a.rows_a * a.K >= ((int64_t)1 << 32)) return launch_gathered_far(a, stream);
  switch (i8_choice(a.M, a.N, a.K, a.offsets == nullptr ? 0 : a.E)) {
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
    default:
      return launch_variant<7, Tile256x256>(a, stream);
  }
}

}  // namespace mxg
