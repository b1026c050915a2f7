// gemm_fp8.hip - E4M3 x E4M3 products with one fp32 scale per row of A and
// 128 columns, and per 128 x 128 block of B, dense and by expert:
//   C[i][j] = out(act(sum_b (sA[i][b] sB[j / 128][b]) p_b[i][j] + bias_j)),
//   p_b = sum_{k in block b} a_ik b_jk.
// The scales of a block are multiplied in fp32, p_b (an MFMA's sum) times that
// is added to the fp32 accumulator by an fma, block after block.
//
// By expert, rows and offsets are as in gemm_int8.hip.
#include "mxg_fp8.h"
#include "mxg_internal.h"

namespace mxg {
namespace {

// 64 x 64 tiles, 4 waves of 32 x 32, a block of 128 k at a time through
// registers.
constexpr int kBM = 64, kBN = 64, kBK = 128;
constexpr int kCus = 256;

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

hipError_t launch_tile(const F8Args& a, hipStream_t stream) {
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
  return launch_tile(a, stream);
}

}  // namespace mxg
